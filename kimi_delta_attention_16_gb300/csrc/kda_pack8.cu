// kda_pack8.cu -- rows stored as e4m3 codes with one power of two per 32 channels, and back.
//
//   e = the smallest exponent with max|x| <= 448 2^e over the block (448 = the largest e4m3 value)
//   code = e4m3(x 2^-e), byte = e + 127;  x ~ code 2^e
//
// The scaling is exact, so the code's own rounding (half a step: 2^-4 relative) is the only one,
// and the packed form does not depend on how the maximum is reduced.  Bound by HBM: 2 + 1 bytes
// per bf16 element, one way.  Four lanes share a block (8 elements each: one 16-byte access of
// bf16, two of fp32) and join their maxima with two shuffles; a thread takes kRows rows of the
// same columns at once to keep enough loads in flight.
//
// Measured, 8,192 x 12,288 bf16: packing 55 us (5.5 TB/s, the integer pipe 53 % busy: maxima, widening, conversions),
// unpacking 46 us (6.5 TB/s).  Two rows per thread and six blocks: 59 and 50 us; eight rows: 60 and 56.
#include "kda_block.cuh"

namespace kda {

namespace {

constexpr int kThreads = 256;
constexpr int kElems = 8;  // elements per thread and row
constexpr int kRows = 4;   // rows per thread

// The scale byte (e + 127) of a block whose largest finite magnitude has these fp32 bits: the exponent, one
// more where the mantissa is above 1.75 (448 = 1.75 * 2^8), and never below that of 2^-126.
__device__ __forceinline__ uint32_t scale_byte(uint32_t bits) {
    const int e = (int)((bits + 0x1fffffu) >> 23) - 8;
    return e < 1 ? 1u : (uint32_t)e;
}

// Largest magnitude among a thread's elements, as fp32 bits (magnitudes order as integers), not finite
// where an element is.
template <int W, int K> __device__ __forceinline__ uint32_t abs_max(const Raw<float, W> (&r)[K]) {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < K; ++i)
#pragma unroll
        for (int j = 0; j < W; ++j) m = max(m, r[i].w[j] & 0x7fffffffu);
    return m;
}
template <int W, int K> __device__ __forceinline__ uint32_t abs_max(const Raw<bf16, W> (&r)[K]) {
    constexpr int kWords = W >= 2 ? W / 2 : 1;
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < K; ++i)
#pragma unroll
        for (int j = 0; j < kWords; ++j) m = __vmaxu2(m, r[i].w[j] & 0x7fff7fffu);
    return max(m << 16, m & 0xffff0000u);
}

// Two values (already divided by the block's power of two, at most 448 in magnitude) as codes; NaN and
// infinities become the NaN code.
__device__ __forceinline__ uint32_t to_e4m3x2(float lo, float hi) {
    unsigned short r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}

template <typename T>
__global__ void __launch_bounds__(kThreads, sizeof(T) == 2 ? 4 : 3) k_pack8(const T* __restrict__ x, int64_t xs, int64_t M, int C,
                                                    uint8_t* __restrict__ codes, uint8_t* __restrict__ scales) {
    constexpr int W = 16 / (int)sizeof(T);
    const int nb = (C + KDA_PACK8_BLOCK - 1) / KDA_PACK8_BLOCK;
    const int c0 = (blockIdx.x * blockDim.x + threadIdx.x) * kElems;
    const int n = c0 < C ? (C - c0 < kElems ? C - c0 : kElems) : 0;  // elements of this thread inside the row
    const int64_t tile = (int64_t)blockDim.y * kRows;
    for (int64_t base = blockIdx.y * tile; base < M; base += gridDim.y * tile) {  // the same for the whole block
        const int64_t r0 = base + threadIdx.y * kRows;
        const int rows = n == 0 || r0 >= M ? 0 : M - r0 < kRows ? (int)(M - r0) : kRows;  // this thread's
        const T* src = x + r0 * xs + c0;
        uint8_t *dst = codes + r0 * C + c0, *sdst = scales + r0 * nb + c0 / KDA_PACK8_BLOCK;
        Raw<T, W> raw[kRows][kElems / W];
#pragma unroll
        for (int q = 0; q < kRows; ++q) {
#pragma unroll
            for (int i = 0; i < kElems / W; ++i)
                if (q < rows && (W == kElems || i * W < n)) raw[q][i].load(src + i * W); else raw[q][i].zero();
            src += xs;
        }
#pragma unroll
        for (int q = 0; q < kRows; ++q, dst += C, sdst += nb) {
            float v[kElems];
#pragma unroll
            for (int i = 0; i < kElems / W; ++i) {
                float t[W];
                unraw(raw[q][i], t);
#pragma unroll
                for (int j = 0; j < W; ++j) v[i * W + j] = t[j];
            }
            uint32_t amax = abs_max(raw[q]);
            if (amax >= 0x7f800000u) {  // rare: infinities turn into NaN, and neither counts
                amax = 0;
#pragma unroll
                for (int j = 0; j < kElems; ++j) {
                    const uint32_t m = __float_as_uint(v[j]) & 0x7fffffffu;
                    if (m >= 0x7f800000u) v[j] = __uint_as_float(0x7fffffffu); else amax = max(amax, m);
                }
            }
            amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
            amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
            if (q >= rows) continue;  // every lane comes to the shuffles
            const uint32_t byte = scale_byte(amax);
            const f2 inv = f2_dup(__uint_as_float((254u - byte) << 23));  // 2^-e
            uint32_t two[kElems / 2];
#pragma unroll
            for (int i = 0; i < kElems / 2; ++i) {
                const f2 s = mul2(f2_of(v[2 * i], v[2 * i + 1]), inv);
                two[i] = to_e4m3x2(f2_lo(s), f2_hi(s));
            }
#pragma unroll
            for (int i = 0; i < kElems / 4; ++i) two[i] = two[2 * i] | (two[2 * i + 1] << 16);
            if constexpr (W == kElems) {  // C is a multiple of W, so a row's codes start on a W-byte boundary
                *reinterpret_cast<uint2*>(dst) = make_uint2(two[0], two[1]);
            } else {
#pragma unroll
                for (int i = 0; i < kElems / 4; ++i)
                    if (i * 4 < n) reinterpret_cast<uint32_t*>(dst)[i] = two[i];
            }
            if ((threadIdx.x & 3) == 0) *sdst = (uint8_t)byte;
        }
    }
}

template <typename T>
__global__ void __launch_bounds__(kThreads, 4) k_unpack8(const uint8_t* __restrict__ codes,
                                                      const uint8_t* __restrict__ scales, int64_t M, int C,
                                                      T* __restrict__ x, int64_t xs) {
    constexpr int W = 16 / (int)sizeof(T);
    const int nb = (C + KDA_PACK8_BLOCK - 1) / KDA_PACK8_BLOCK;
    const int c0 = (blockIdx.x * blockDim.x + threadIdx.x) * kElems;
    const int n = c0 < C ? (C - c0 < kElems ? C - c0 : kElems) : 0;
    if (n == 0) return;
    const int64_t tile = (int64_t)blockDim.y * kRows;
    for (int64_t base = blockIdx.y * tile; base < M; base += gridDim.y * tile) {  // the same for the whole block
        const int64_t r0 = base + threadIdx.y * kRows;
        const int rows = r0 >= M ? 0 : M - r0 < kRows ? (int)(M - r0) : kRows;  // this thread's
        const uint8_t *src = codes + r0 * C + c0, *ssrc = scales + r0 * nb + c0 / KDA_PACK8_BLOCK;
        T* dst = x + r0 * xs + c0;
        Raw<uint8_t, W> raw[kRows][kElems / W];
        uint32_t sc[kRows];
#pragma unroll
        for (int q = 0; q < kRows; ++q) {
            sc[q] = q < rows ? (uint32_t)__ldg(ssrc) : 127u;
#pragma unroll
            for (int i = 0; i < kElems / W; ++i)
                if (q < rows && (W == kElems || i * W < n)) raw[q][i].load(src + i * W); else raw[q][i].zero();
            src += C;
            ssrc += nb;
        }
#pragma unroll
        for (int q = 0; q < kRows; ++q) {
            if (q >= rows) break;
#pragma unroll
            for (int i = 0; i < kElems / W; ++i) {
                float t[W];
                unraw8(raw[q][i], scale_of_byte(sc[q]), t);
                if (W == kElems || i * W < n) store_row(dst + i * W, t);
            }
            dst += xs;
        }
    }
}

// Rows that allow no wide accesses (an odd number of channels above all): a warp takes eight blocks of 32 channels of
// one row, a lane one element of each, so that every access of the warp is one piece of the row (8,192 x 7,167 bf16:
// 61 us packing, 48 unpacking; with the eight neighbours of a lane one by one, 70 and 146).
template <typename T>
__global__ void __launch_bounds__(kThreads) k_pack8_single(const T* __restrict__ x, int64_t xs, int64_t M, int C,
                                                           uint8_t* __restrict__ codes, uint8_t* __restrict__ scales) {
    const int lane = threadIdx.x & 31, nb = (C + KDA_PACK8_BLOCK - 1) / KDA_PACK8_BLOCK;
    for (int64_t r = (int64_t)blockIdx.x * (kThreads / 32) + threadIdx.x / 32; r < M; r += (int64_t)gridDim.x * (kThreads / 32))
        for (int b0 = blockIdx.y * kElems; b0 < nb; b0 += gridDim.y * kElems) {
            const int c0 = b0 * KDA_PACK8_BLOCK + lane;
            const T* src = x + r * xs + c0;
            uint8_t *dst = codes + r * C + c0, *sdst = scales + r * nb + b0;
            Raw<T, 1> raw[kElems];
#pragma unroll
            for (int i = 0; i < kElems; ++i)
                if (c0 + i * 32 < C) raw[i].load(src + i * 32); else raw[i].zero();
#pragma unroll
            for (int i = 0; i < kElems; ++i) {
                if (b0 + i >= nb) break;  // the same for the whole warp
                float v[1];
                unraw(raw[i], v);
                uint32_t m = __float_as_uint(v[0]) & 0x7fffffffu;
                if (m >= 0x7f800000u) {  // infinities turn into NaN, and neither counts
                    v[0] = __uint_as_float(0x7fffffffu);
                    m = 0;
                }
                const uint32_t byte = scale_byte(__reduce_max_sync(0xffffffffu, m));
                const uint32_t code = to_e4m3x2(v[0] * __uint_as_float((254u - byte) << 23), 0.f);
                if (c0 + i * 32 < C) dst[i * 32] = (uint8_t)code;
                if (lane == 0) sdst[i] = (uint8_t)byte;
            }
        }
}
template <typename T>
__global__ void __launch_bounds__(kThreads) k_unpack8_single(const uint8_t* __restrict__ codes,
                                                             const uint8_t* __restrict__ scales, int64_t M, int C,
                                                             T* __restrict__ x, int64_t xs) {
    const int lane = threadIdx.x & 31, nb = (C + KDA_PACK8_BLOCK - 1) / KDA_PACK8_BLOCK;
    for (int64_t r = (int64_t)blockIdx.x * (kThreads / 32) + threadIdx.x / 32; r < M; r += (int64_t)gridDim.x * (kThreads / 32))
        for (int b0 = blockIdx.y * kElems; b0 < nb; b0 += gridDim.y * kElems) {
            const int c0 = b0 * KDA_PACK8_BLOCK + lane;
            const uint8_t *src = codes + r * C + c0, *ssrc = scales + r * nb + b0;
            T* dst = x + r * xs + c0;
            Raw<uint8_t, 1> raw[kElems];
            uint32_t sc[kElems];
#pragma unroll
            for (int i = 0; i < kElems; ++i) {
                raw[i].zero();
                sc[i] = 127u;
                if (c0 + i * 32 < C) {
                    raw[i].load(src + i * 32);
                    sc[i] = (uint32_t)__ldg(ssrc + i);
                }
            }
#pragma unroll
            for (int i = 0; i < kElems; ++i) {
                float v[1];
                unraw8(raw[i], scale_of_byte(sc[i]), v);
                if (c0 + i * 32 < C) store_row(dst + i * 32, v);
            }
        }
}

// Rows of `stride` elements at p allow 16-byte accesses of T, and rows of C codes the matching ones.
template <typename T> bool vec_ok(const void* p, int64_t stride, const uint8_t* codes, int C) {
    constexpr int W = 16 / (int)sizeof(T);
    return reinterpret_cast<uintptr_t>(p) % 16 == 0 && stride % W == 0 && C % W == 0 &&
           reinterpret_cast<uintptr_t>(codes) % 8 == 0;
}

// Narrow rows share a block: x = the threads of a row (a power of two, at least the four of one
// 32-channel block), y = rows.
dim3 block_of(int C) {
    int x = 4;
    while (x < kThreads && x * kElems < C) x *= 2;
    return dim3(x, kThreads / x);
}
dim3 grid_of(int64_t M, int C) {
    const dim3 b = block_of(C);
    const int64_t rows = (M + b.y * kRows - 1) / (b.y * kRows);
    return dim3((unsigned)((C + b.x * kElems - 1) / (b.x * kElems)), (unsigned)(rows < 65535 ? rows : 65535));
}

// One row per warp, chunks of eight blocks of channels.
dim3 grid_single(int64_t M, int C) {
    const int64_t rows = (M + kThreads / 32 - 1) / (kThreads / 32), chunks = (C + kElems * 32 - 1) / (kElems * 32);
    return dim3((unsigned)(rows < 0x7fffffff ? rows : 0x7fffffff), (unsigned)(chunks < 65535 ? chunks : 65535));
}

}  // namespace

cudaError_t launch_pack8(const void* x, int64_t x_stride, kda_dtype dt, int64_t M, int C, uint8_t* codes,
                         uint8_t* scales, cudaStream_t s) {
    const dim3 g = grid_of(M, C), b = block_of(C);
    if (dt == KDA_BF16) {
        const bf16* p = static_cast<const bf16*>(x);
        if (vec_ok<bf16>(x, x_stride, codes, C)) k_pack8<bf16><<<g, b, 0, s>>>(p, x_stride, M, C, codes, scales);
        else k_pack8_single<bf16><<<grid_single(M, C), kThreads, 0, s>>>(p, x_stride, M, C, codes, scales);
    } else {
        const float* p = static_cast<const float*>(x);
        if (vec_ok<float>(x, x_stride, codes, C)) k_pack8<float><<<g, b, 0, s>>>(p, x_stride, M, C, codes, scales);
        else k_pack8_single<float><<<grid_single(M, C), kThreads, 0, s>>>(p, x_stride, M, C, codes, scales);
    }
    return cudaGetLastError();
}

cudaError_t launch_unpack8(const uint8_t* codes, const uint8_t* scales, int64_t M, int C, void* x, int64_t x_stride,
                           kda_dtype dt, cudaStream_t s) {
    const dim3 g = grid_of(M, C), b = block_of(C);
    if (dt == KDA_BF16) {
        bf16* p = static_cast<bf16*>(x);
        if (vec_ok<bf16>(x, x_stride, codes, C)) k_unpack8<bf16><<<g, b, 0, s>>>(codes, scales, M, C, p, x_stride);
        else k_unpack8_single<bf16><<<grid_single(M, C), kThreads, 0, s>>>(codes, scales, M, C, p, x_stride);
    } else {
        float* p = static_cast<float*>(x);
        if (vec_ok<float>(x, x_stride, codes, C)) k_unpack8<float><<<g, b, 0, s>>>(codes, scales, M, C, p, x_stride);
        else k_unpack8_single<float><<<grid_single(M, C), kThreads, 0, s>>>(codes, scales, M, C, p, x_stride);
    }
    return cudaGetLastError();
}

}  // namespace kda
