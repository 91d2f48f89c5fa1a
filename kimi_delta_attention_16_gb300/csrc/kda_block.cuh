// kda_block.cuh -- internal launch declarations and device helpers of the operators around the
// layer (kda_norm.cu, kda_pack8.cu, kda_ssm_*.cu).  Not part of the public ABI.
#pragma once

#include "kda_internal.cuh"

namespace kda {

// ------------------------------------------------------------------ rows of W elements per access
// W consecutive elements of a row as they lie in memory: W * sizeof(T) bytes, 16 when the layout
// allows vectors, one element otherwise.  load() only moves bytes, so several can be in flight
// before the first conversion.
template <typename T, int W> struct alignas(W * sizeof(T)) Raw {
    static constexpr int kBytes = W * (int)sizeof(T);
    static_assert(kBytes == 16 || kBytes == 8 || kBytes == 4 || kBytes == 2 || kBytes == 1, "access width");
    uint32_t w[kBytes >= 4 ? kBytes / 4 : 1];
    __device__ __forceinline__ void load(const T* p) {
        if constexpr (kBytes == 16) {
            const uint4 u = __ldg(reinterpret_cast<const uint4*>(p));
            w[0] = u.x; w[1] = u.y; w[2] = u.z; w[3] = u.w;
        } else if constexpr (kBytes == 8) {
            const uint2 u = __ldg(reinterpret_cast<const uint2*>(p));
            w[0] = u.x; w[1] = u.y;
        } else if constexpr (kBytes == 4) {
            w[0] = __ldg(reinterpret_cast<const unsigned int*>(p));
        } else if constexpr (kBytes == 2) {
            w[0] = __ldg(reinterpret_cast<const unsigned short*>(p));
        } else {
            w[0] = __ldg(reinterpret_cast<const unsigned char*>(p));
        }
    }
    __device__ __forceinline__ void zero() {
#pragma unroll
        for (int i = 0; i < (kBytes >= 4 ? kBytes / 4 : 1); ++i) w[i] = 0;
    }
};
template <int W> __device__ __forceinline__ void unraw(const Raw<float, W>& r, float (&v)[W]) {
#pragma unroll
    for (int i = 0; i < W; ++i) v[i] = __uint_as_float(r.w[i]);
}
template <int W> __device__ __forceinline__ void unraw(const Raw<bf16, W>& r, float (&v)[W]) {
    if constexpr (W == 1) {
        v[0] = __uint_as_float(r.w[0] << 16);
    } else {
#pragma unroll
        for (int i = 0; i < W / 2; ++i) {
            v[2 * i] = __uint_as_float(r.w[i] << 16);
            v[2 * i + 1] = __uint_as_float(r.w[i] & 0xffff0000u);
        }
    }
}
// The same as fp32 pairs; one element makes a pair with zero.
template <typename T, int W> __device__ __forceinline__ void unraw2(const Raw<T, W>& r, f2 (&v)[(W + 1) / 2]) {
    float t[W];
    unraw(r, t);
#pragma unroll
    for (int i = 0; i < (W + 1) / 2; ++i) v[i] = f2_of(t[2 * i], 2 * i + 1 < W ? t[2 * i + 1] : 0.f);
}
template <int W> __device__ __forceinline__ void store_row(float* p, const float (&v)[W]) {
    if constexpr (W == 4) {
        *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
    } else {
        static_assert(W == 1, "fp32 rows: 4 or 1 elements");
        *p = v[0];
    }
}
template <int W> __device__ __forceinline__ void store_row(bf16* p, const float (&v)[W]) {
    if constexpr (W == 8) {
        store8(p, v);
    } else if constexpr (W == 4) {
        *reinterpret_cast<uint2*>(p) = make_uint2(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]));
    } else {
        static_assert(W == 1, "bf16 rows: 8, 4 or 1 elements");
        *p = __float2bfloat16_rn(v[0]);
    }
}
template <typename T, int W> __device__ __forceinline__ void store_row2(T* p, const f2 (&v)[(W + 1) / 2]) {
    float t[W];
#pragma unroll
    for (int i = 0; i < W; ++i) t[i] = i & 1 ? f2_hi(v[i / 2]) : f2_lo(v[i / 2]);
    store_row(p, t);
}
// fp32 parameters (weights, biases) for W consecutive channels; 16-byte accesses when W allows.
template <int W> __device__ __forceinline__ void load_param(const float* p, float (&v)[W]) {
    if constexpr (W % 4 == 0) {
#pragma unroll
        for (int i = 0; i < W / 4; ++i) {
            const float4 f = __ldg(reinterpret_cast<const float4*>(p) + i);
            v[4 * i] = f.x; v[4 * i + 1] = f.y; v[4 * i + 2] = f.z; v[4 * i + 3] = f.w;
        }
    } else {
#pragma unroll
        for (int i = 0; i < W; ++i) v[i] = __ldg(p + i);
    }
}

// ------------------------------------------------------------------ activations
// Sigmoid and SiLU from the hardware's exponential and reciprocal, without the range checks of the library
// forms: e^-x overflows to a sigmoid of 0, as it should.  In units of 2^-24, relative: the exponential 4, the
// reciprocal 2, and for negative x the rounding of the exponent x log2 e, |x| units (10 at -10, where SiLU has
// 5e-5 of x left).  The convolution and the gates take it so: bf16 rows round by 2^16 units, fp32 rows carry
// these, and correcting the exponent would cost a guard against infinities in every token.
__device__ __forceinline__ float rcp_hw(float x) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float sigmoid(float x) { return rcp_hw(1.f + exp2_hw(-kLog2e * x)); }
__device__ __forceinline__ float silu(float x) { return x * sigmoid(x); }
__device__ __forceinline__ f2 exp2_2(f2 x) { return f2_of(exp2_hw(f2_lo(x)), exp2_hw(f2_hi(x))); }
__device__ __forceinline__ f2 sigmoid2(f2 x) {
    const f2 d = add2(exp2_2(mul2(x, f2_dup(-kLog2e))), f2_dup(1.f));
    return f2_of(rcp_hw(f2_lo(d)), rcp_hw(f2_hi(d)));
}

// ------------------------------------------------------------------ asynchronous copies to shared memory
__device__ __forceinline__ void cp_async16(void* dst, const void* src) {
    const uint32_t d = (uint32_t)__cvta_generic_to_shared(dst);
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(d), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N> __device__ __forceinline__ void cp_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }
// All W elements of an access (4, 8 or 16 bytes).
template <typename T, int W> __device__ __forceinline__ void cp_async_raw(Raw<T, W>* dst, const T* src) {
    constexpr int n = Raw<T, W>::kBytes;
    const uint32_t d = (uint32_t)__cvta_generic_to_shared(dst);
    if constexpr (n == 16)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(d), "l"(src) : "memory");
    else
        asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(d), "l"(src), "n"(n) : "memory");
}

// ------------------------------------------------------------------ e4m3 in blocks of 32
// Byte s stands for 2^(s - 127), s >= 1 (a normal fp32 number).
__device__ __forceinline__ float scale_of_byte(uint32_t s) { return __uint_as_float(s << 23); }
// Two codes (low byte first) as fp32 values before the block's scale: by way of fp16, which holds
// every e4m3 value exactly.
__device__ __forceinline__ void e4m3x2_to_f(uint32_t two, float& lo, float& hi) {
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((unsigned short)two));
    asm("{.reg .f16 a, b; mov.b32 {a, b}, %2; cvt.f32.f16 %0, a; cvt.f32.f16 %1, b;}"
        : "=f"(lo), "=f"(hi) : "r"(h));
}
template <int W> __device__ __forceinline__ void unraw(const Raw<uint8_t, W>& r, float (&v)[W]) {  // codes, unscaled
    if constexpr (W == 1) {
        float unused;
        e4m3x2_to_f(r.w[0] & 0xffu, v[0], unused);
    } else {
#pragma unroll
        for (int i = 0; i < W / 2; ++i)
            e4m3x2_to_f((r.w[i / 2] >> (16 * (i & 1))) & 0xffffu, v[2 * i], v[2 * i + 1]);
    }
}
template <int W> __device__ __forceinline__ void unraw8(const Raw<uint8_t, W>& r, float scale, float (&v)[W]) {
    unraw(r, v);
#pragma unroll
    for (int i = 0; i < W; ++i) v[i] *= scale;
}

// ------------------------------------------------------------------ sums in a fixed order
// Column sums of part [rows][W] fp32: 32 columns per block, the rows dealt to 32 warps and joined in
// a fixed order, so the result depends on nothing but rows, W and the values.  put(column, sum).
template <typename Put>
__global__ void __launch_bounds__(1024) k_column_sum(const float* __restrict__ part, int64_t rows, int64_t W, Put put) {
    __shared__ float sm[32][33];
    const int64_t c = (int64_t)blockIdx.x * 32 + threadIdx.x;
    float s = 0.f;
    if (c < W) {
#pragma unroll 4
        for (int64_t g = threadIdx.y; g < rows; g += 32) s += part[g * W + c];
    }
    sm[threadIdx.y][threadIdx.x] = s;
    __syncthreads();
    if (threadIdx.y || c >= W) return;
    s = 0.f;
#pragma unroll
    for (int k = 0; k < 32; ++k) s += sm[k][threadIdx.x];
    put(c, s);
}
// Few rows of many columns: one thread per column (29 rows of 65,536: 3 us, against 12 with a warp row per part).
template <typename Put>
__global__ void __launch_bounds__(256) k_column_sum_flat(const float* __restrict__ part, int rows, int64_t W, Put put) {
    const int64_t c = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (c >= W) return;
    float s = 0.f;
#pragma unroll 8
    for (int g = 0; g < rows; ++g) s += part[g * W + c];
    put(c, s);
}
template <typename Put>
cudaError_t launch_column_sum(const float* part, int64_t rows, int64_t W, Put put, cudaStream_t s) {
    if (rows <= 64 && W >= 16384) {
        k_column_sum_flat<<<(unsigned)((W + 255) / 256), 256, 0, s>>>(part, (int)rows, W, put);
        return cudaGetLastError();
    }
    k_column_sum<<<(unsigned)((W + 31) / 32), dim3(32, 32), 0, s>>>(part, rows, W, put);
    return cudaGetLastError();
}

// ------------------------------------------------------------------ packed sequences
// The sequence that holds token t: the last n in [0, N) with cu[n] <= t (cu[n + 1] > t when cu is
// consistent, so empty sequences are passed over).  Always in range.
__device__ __forceinline__ int seq_of(const int32_t* __restrict__ cu, int N, int64_t t) {
    int lo = 0, hi = N - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if ((int64_t)cu[mid] <= t) lo = mid; else hi = mid - 1;
    }
    return lo;
}

// A copy of cu in shared memory where it fits: looking a token up there costs no chain of memory
// latencies.  Every thread of the block calls it; it ends with a barrier.
constexpr int kStagedCu = 512;
__device__ __forceinline__ const int32_t* stage_cu(const int32_t* __restrict__ cu, int N, int32_t (&shared)[kStagedCu]) {
    const int t = threadIdx.y * blockDim.x + threadIdx.x, nt = blockDim.x * blockDim.y;
    if (N < kStagedCu)
        for (int i = t; i <= N; i += nt) shared[i] = cu[i];
    __syncthreads();
    return N < kStagedCu ? shared : cu;
}

// ------------------------------------------------------------------ launchers (arguments validated by the caller)
// dst[n] = src[n] (zeros when src is NULL) for every sequence of no tokens, `per` bytes each (a
// multiple of 2): what a kernel over tokens never reaches.
cudaError_t launch_empty_sequences(const int32_t* cu, int N, const void* src, void* dst, int64_t per, cudaStream_t s);

cudaError_t launch_ssm_conv(const kda_ssm_conv_args& a, cudaStream_t s);
cudaError_t launch_ssm_conv_step(const kda_ssm_conv_args& a, cudaStream_t s);
struct ConvBackwardPlan {
    int run;        // tokens per thread
    int64_t rows;   // partial sums of dw and dbias
    size_t workspace;
};
ConvBackwardPlan conv_backward_plan(const kda_ssm_conv_args& f);
cudaError_t launch_ssm_conv_backward(const kda_ssm_conv_backward_args& a, const ConvBackwardPlan& p, cudaStream_t s);

// Pieces of the packed token axis that the scan runs side by side, and where the workspace holds
// their states [pieces][C][Nst] and sums of delta [pieces][C].
struct ScanPlan {
    int64_t piece;   // tokens per piece (a multiple of the tile)
    int pieces;
    size_t sums;     // byte offset
    size_t workspace;
};
ScanPlan scan_plan(const kda_ssm_args& a);
cudaError_t launch_ssm_scan(const kda_ssm_args& a, const ScanPlan& p, cudaStream_t s);
cudaError_t launch_ssm_step(const kda_ssm_args& a, cudaStream_t s);

// The scan's gradients: pieces of the token axis and the byte offsets of the workspace's parts.
struct SsmBackwardPlan {
    int64_t piece;
    int pieces;
    size_t fwd, rev;      // [pieces][C][Nst]: states at the pieces' starts; gradients that enter from the right
    size_t fsum, rsum;    // [pieces][C]: sums of delta
    size_t ckpt;          // [ceil(T / 4)][C][Nst]: the state in front of every fourth token
    size_t pa;            // [pieces][C][Nst]: parts of dA
    size_t pd;            // [pieces * rows][2][C]: parts of dD and ddt_bias
    size_t pbc;           // [G * blocks][T][2 Nst]: parts of dB and dC
    size_t workspace;
};
SsmBackwardPlan ssm_backward_plan(const kda_ssm_args& f);
cudaError_t launch_ssm_backward(const kda_ssm_backward_args& a, const SsmBackwardPlan& p, cudaStream_t s);

cudaError_t launch_layer_norm(const kda_norm_args& a, cudaStream_t s);

// How many row blocks kda_layer_norm_backward runs for M rows of C channels: each leaves one
// partial sum of the weight's and the bias's gradient in the workspace.
struct NormBackwardPlan {
    int blocks;
    size_t workspace;  // bytes
};
NormBackwardPlan norm_backward_plan(const kda_norm_backward_args& a);
cudaError_t launch_layer_norm_backward(const kda_norm_backward_args& a, const NormBackwardPlan& p, cudaStream_t s);

cudaError_t launch_pack8(const void* x, int64_t x_stride, kda_dtype dt, int64_t M, int C, uint8_t* codes,
                         uint8_t* scales, cudaStream_t s);
cudaError_t launch_unpack8(const uint8_t* codes, const uint8_t* scales, int64_t M, int C, void* x, int64_t x_stride,
                           kda_dtype dt, cudaStream_t s);

}  // namespace kda
