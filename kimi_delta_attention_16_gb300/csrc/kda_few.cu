// kda_few.cu -- the columns of the products with integer codes (kda_few.cuh): bf16 rows as fp16, each run of 128 under a
// power of two, elements in the order in which codes come out of a word, and the groups' sums of what is stored.  A block
// takes 2,048 values of a row.
#include "kda_few.cuh"

namespace kda {
namespace few {

__global__ void __launch_bounds__(256) k_few_halves(const bf16* __restrict__ x, int64_t xs, bool wide, int K, int group, __half* __restrict__ columns,
                                                    float* __restrict__ factor, float* __restrict__ sums) {
    let_next_kernel_begin();
    const int64_t p = blockIdx.y;
    const int k = (blockIdx.x * 256 + threadIdx.x) * 8;
    const bool in = k < K;  // K is a multiple of 32: a run's 16 lanes may be part full
    uint32_t v[4] = {};
    if (in) {
        const bf16* row = x + p * xs + k;
        if (wide) {
            const uint4 q = *reinterpret_cast<const uint4*>(row);
            v[0] = q.x, v[1] = q.y, v[2] = q.z, v[3] = q.w;
        } else {
            const unsigned short* h = reinterpret_cast<const unsigned short*>(row);
#pragma unroll
            for (int i = 0; i < 4; ++i) v[i] = h[2 * i] | ((uint32_t)h[2 * i + 1] << 16);
        }
    }
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) top = __vmaxu2(top, v[i] & 0x7fff7fffu);
    top = max(top << 16, top & 0xffff0000u);
#pragma unroll
    for (int d = 1; d < 16; d <<= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, d));
    float up, down, r[8];
    run_scale(top >> 23, up, down);
#pragma unroll
    for (int i = 0; i < 4; ++i) r[2 * i] = __uint_as_float(v[i] << 16) * up, r[2 * i + 1] = __uint_as_float(v[i] & 0xffff0000u) * up;
    uint32_t o[4];
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        o[i] = pack_half2(r[i], r[i + 4]);
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&o[i]));
        sum += f.x + f.y;
    }
    for (int d = 1; d < group / 8; d <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
    if (in) {
        *reinterpret_cast<uint4*>(columns + p * K + k) = make_uint4(o[0], o[1], o[2], o[3]);
        if (k % kRun == 0) factor[p * ((K + kRun - 1) / kRun) + k / kRun] = down;
        if (k % group == 0) sums[p * (K / group) + k / group] = kSumOf * sum;
    }
}

cudaError_t launch_halves(const bf16* x, int64_t xs, bool wide, int rows, int K, int group, const Columns& c, cudaStream_t s) {
    return launch_kernel(k_few_halves, dim3((K + 2047) / 2048, rows), 256, 1, 0, false, s, x, xs, wide, K, group, const_cast<__half*>(c.x),
                         const_cast<float*>(c.factor), const_cast<float*>(c.sums));
}

}  // namespace few
}  // namespace kda
