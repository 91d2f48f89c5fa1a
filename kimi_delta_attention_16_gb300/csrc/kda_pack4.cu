// kda_pack4.cu -- weights stored in 4 bits with one scale per group along a row, and back.
//
//   e2m1  32 weights under the smallest power of two 2^e with max|w| <= 6 2^e (6 = the largest e2m1 value);
//         code = e2m1(w 2^-e), scale byte e + 127
//   int4  32, 64 or 128 weights under scale = max|w| / 7, rounded to the scales' type;
//         code = round(w / scale) + 8
//
// Weights are laid out once, so this is plain: four lanes share 32 weights (8 each) and join their maxima by
// shuffles, each writes its 8 codes as one word, the even weight in the low half of a byte.  24,576 x 7,168 bf16:
// e2m1 104 us (4.2 TB/s), back 121; int4 211 (its divisions), back 88.
#include "kda_serve.cuh"

namespace kda {

namespace {

constexpr int kThreads = 256;

template <typename T> __device__ __forceinline__ void load8_any(const T* p, bool wide, float (&v)[8]) {
    if (wide) {
        load8(p, v);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = to_f(p[i]);
    }
}

// Eight values as e2m1 codes, the first one lowest; beyond 6 they become 6.
__device__ __forceinline__ uint32_t e2m1x8(const float (&v)[8]) {
    uint32_t r;
    asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n\tcvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n\tcvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n\t"
        "mov.b32 %0, {b0, b1, b2, b3};\n\t}"
        : "=r"(r) : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]));
    return r;
}

template <typename T, bool E2m1, typename S>
__global__ void __launch_bounds__(kThreads) k_pack4(const T* __restrict__ w, int64_t ws, int64_t rows, int K, int shift, bool wide,
                                                    uint32_t* __restrict__ codes, S* __restrict__ scales) {
    const int words = K / 8;
    const int64_t total = rows * words, step = (int64_t)gridDim.x * kThreads;
    const int lanes = 4 << shift;  // that share a group; a group never leaves its warp, whose words are all inside or all outside
    for (int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x; i - (threadIdx.x & 31) < total; i += step) {
        const bool in = i < total;  // the last warp may be part full: whole groups all the same
        const int64_t row = in ? i / words : 0;
        const int q = in ? (int)(i - row * words) : 0;
        float v[8] = {};
        if (in) load8_any(w + row * ws + 8 * q, wide, v);
        uint32_t top = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j) top = max(top, __float_as_uint(v[j]) & 0x7fffffffu);
        for (int d = 1; d < lanes; d <<= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, d));
        top = min(top, 0x7f7fffffu);
        uint32_t word = 0;
        const bool first = (threadIdx.x & (lanes - 1)) == 0;
        if constexpr (E2m1) {
            // the exponent, one more where the mantissa is above 1.5 (6 = 1.5 * 4), and never below that of 2^-126
            const int b = max((int)((top + 0x3fffffu) >> 23) - 2, 1);
            const uint32_t inv = 254u - (uint32_t)b;
            const float down = __uint_as_float(inv << 23);  // b is at most 253
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] *= down;
            word = e2m1x8(v);
            if (in && first) scales[i >> 2] = (S)b;
        } else {
            const S s = from_f<S>(__uint_as_float(top) / 7.0f);
            const float f = to_f(s);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float c = f > 0.f ? fminf(fmaxf(rintf(v[j] / f), -8.f), 7.f) : 0.f;
                word |= (uint32_t)((int)c + 8) << (4 * j);
            }
            if (in && first) scales[i >> (2 + shift)] = s;
        }
        if (in) codes[i] = word;
    }
}

template <typename T, bool E2m1, typename S>
__global__ void __launch_bounds__(kThreads) k_unpack4(T* __restrict__ w, int64_t ws, int64_t rows, int K, int shift, bool wide,
                                                      const uint32_t* __restrict__ codes, const S* __restrict__ scales) {
    const int words = K / 8;
    const int64_t total = rows * words, step = (int64_t)gridDim.x * kThreads;
    for (int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x; i < total; i += step) {
        const int64_t row = i / words;
        const int q = (int)(i - row * words);
        const uint32_t word = codes[i];
        float v[8];
        if constexpr (E2m1) {
            const float s = __uint_as_float((uint32_t)scales[i >> 2] << 23);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const uint32_t c = word >> (4 * j);
                // sign, two bits of exponent, one of mantissa; no implicit one at exponent 0
                const float m = (c & 6u) ? __uint_as_float(((126u + ((c >> 1) & 3u)) << 23) | ((c & 1u) << 22)) : 0.5f * (c & 1u);
                v[j] = ((c & 8u) ? -m : m) * s;
            }
        } else {
            const float s = to_f(scales[i >> (2 + shift)]);
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] = (float)((int)((word >> (4 * j)) & 15u) - 8) * s;
        }
        T* p = w + row * ws + 8 * q;
        if (wide) {
            store8(p, v);
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) p[j] = from_f<T>(v[j]);
        }
    }
}

template <typename T, bool E2m1, typename S> cudaError_t launch(const kda_pack4_args& a, bool pack, cudaStream_t s) {
    const int64_t total = a.rows * (a.K / 8);
    const int blocks = (int)(total / kThreads < 152 * 16 ? (total + kThreads - 1) / kThreads : 152 * 16);
    const int64_t ws = a.w_stride ? a.w_stride : a.K;
    const bool wide = reinterpret_cast<uintptr_t>(a.w) % 16 == 0 && (ws * sizeof(T)) % 16 == 0;
    uint32_t* codes = reinterpret_cast<uint32_t*>(a.codes);
    if (pack)
        k_pack4<T, E2m1, S><<<blocks, kThreads, 0, s>>>(static_cast<const T*>(a.w), ws, a.rows, a.K, group_shift(a.group), wide, codes,
                                                        static_cast<S*>(a.scales));
    else
        k_unpack4<T, E2m1, S><<<blocks, kThreads, 0, s>>>(static_cast<T*>(a.w), ws, a.rows, a.K, group_shift(a.group), wide, codes,
                                                          static_cast<const S*>(a.scales));
    return cudaGetLastError();
}

template <typename T> cudaError_t launch_as(const kda_pack4_args& a, bool pack, cudaStream_t s) {
    if (a.format == KDA_WEIGHT_E2M1) return launch<T, true, uint8_t>(a, pack, s);
    return a.scale_dtype == KDA_BF16 ? launch<T, false, bf16>(a, pack, s) : launch<T, false, float>(a, pack, s);
}

}  // namespace

cudaError_t launch_pack4(const kda_pack4_args& a, cudaStream_t s) {
    return a.w_dtype == KDA_BF16 ? launch_as<bf16>(a, true, s) : launch_as<float>(a, true, s);
}
cudaError_t launch_unpack4(const kda_pack4_args& a, cudaStream_t s) {
    return a.w_dtype == KDA_BF16 ? launch_as<bf16>(a, false, s) : launch_as<float>(a, false, s);
}

}  // namespace kda
