// kda_few_tc.cu -- the columns of the block-scaled products (kda_few_tc.cuh): bf16 rows as digits.  A block takes 2,048
// values of a row; a few microseconds beside the first reads of megabytes of weights.
#include "kda_few_tc.cuh"

namespace kda {
namespace fewtc {

__global__ void __launch_bounds__(256) k_few_digits(const bf16* __restrict__ x, int64_t xs, bool wide, const int* __restrict__ of, int per, int K,
                                                    uint8_t* __restrict__ digits, uint8_t* __restrict__ scales) {
    if (of) few::wait_for_kernel_before();  // the lists
    few::let_next_kernel_begin();           // the products' kernel may read lists and weights
    const int64_t p = blockIdx.y;
    const int k = (blockIdx.x * 256 + threadIdx.x) * 8;
    const bool in = k < K;  // K is a multiple of 32: four lanes at a time
    float r[8] = {};
    if (in) {
        const bf16* row = x + (int64_t)(of ? of[p] / per : (int)p) * xs + k;
        if (wide) {
            load8(row, r);
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) r[i] = to_f(row[i]);
        }
    }
    uint32_t top = largest_of_32(r);
    // Values that lose digits matter where the whole row is as small: then their scale is NaN, which sends the row's sums
    // to direct().  Hardly ever a row is looked through for that.
    const bool tiny = top > 0 && top < kLowestTop;
    if (__syncthreads_or(tiny)) {
        bool normal = false;
        const bf16* row = x + (int64_t)(of ? of[p] / per : (int)p) * xs;
        for (int i = threadIdx.x; i < K; i += 256) normal = normal || fabsf(to_f(row[i])) >= 0x1p-80f;
        if (!__syncthreads_or(normal) && tiny) top = 0x7f800000u;
    }
    put_digits(r, top, in, p, k, K, digits, scales);
}

cudaError_t launch_digits(const bf16* x, int64_t xs, bool wide, const int* of, int per, int tokens, int K, uint8_t* digits, uint8_t* scales,
                          cudaStream_t s) {
    return few::launch_kernel(k_few_digits, dim3((K + 2047) / 2048, tokens), 256, 1, 0, of != nullptr, s, x, xs, wide, of, per, K, digits, scales);
}

// bf16 rows as they are, dense: token p is row of[p] / per of x.
__global__ void __launch_bounds__(256) k_few_rows(const bf16* __restrict__ x, int64_t xs, bool wide, const int* __restrict__ of, int per, int K,
                                                  bf16* __restrict__ rows) {
    few::wait_for_kernel_before();  // the lists
    few::let_next_kernel_begin();
    const int64_t p = blockIdx.y;
    const int k = (blockIdx.x * 256 + threadIdx.x) * 8;  // K is a multiple of 8
    if (k >= K) return;
    const bf16* row = x + (int64_t)(of[p] / per) * xs + k;
    bf16* to = rows + p * K + k;
    if (wide) {
        *reinterpret_cast<uint4*>(to) = *reinterpret_cast<const uint4*>(row);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) to[i] = row[i];
    }
}

cudaError_t launch_rows(const bf16* x, int64_t xs, bool wide, const int* of, int per, int tokens, int K, bf16* rows, cudaStream_t s) {
    return few::launch_kernel(k_few_rows, dim3((K + 2047) / 2048, tokens), 256, 1, 0, true, s, x, xs, wide, of, per, K, rows);
}

}  // namespace fewtc
}  // namespace kda
