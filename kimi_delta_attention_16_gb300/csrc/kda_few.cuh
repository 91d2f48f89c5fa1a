// kda_few.cuh -- products of a weight matrix [rows][K] with a few columns (tokens), for weights in
// 4 bits or bf16: what the 4-bit projections (kda_gemm4.cu) and the experts (kda_moe.cu) share.
//
// Bound by the weights' bytes: every weight is read once and used for at most 8 NT columns.  A CTA
// takes 128 rows, a warp 16 of them, on mma.sync (m16n8k16, fp32 accumulation: an instruction whose
// narrow side is 8 columns fits a few tokens, where a tcgen05 tile of 128 x N would spend its time on
// feeding codes that registers have to widen first).  K is split over the CTAs of a cluster, which
// join their parts through distributed shared memory in the order of their ranks.
//
// 4-bit codes go through cp.async into a ring of stages of each warp's own (16 rows x 128 bytes, no
// barrier among warps), are widened to fp16 in registers, exactly, and multiply columns held in
// shared memory as fp16.  Each run of 256 elements of a column is brought to 2^14..2^15 by a power of
// two first: that is exact for a bf16 element down to 2^-28 of its run's largest and off by at most
// 2^-40 of the largest below that, less than an fp32 sum would keep.  A group's product (32 weights
// under one scale) is a sum of two instructions from zero, multiplied by the weights' scale in fp32
// when it is added up, so scales are never rounded.  bf16 weights multiply bf16 columns.
// fp32 columns (the experts' hidden values) are split into two fp16 or three bf16 terms of a column
// each, added up at the end.
#pragma once

#include <cooperative_groups.h>
#include <cuda_fp16.h>

#include <utility>

#include "kda_internal.cuh"

namespace kda {
namespace few {

constexpr int kThreads = 256, kWarps = 8;
constexpr int kTileRows = 128;               // rows of weights per CTA
constexpr int kChunk = 256;                  // elements of a column under one power of two
constexpr int kRowStage = 128;               // bytes of a row per stage
constexpr int kWarpStage = 16 * kRowStage;   // bytes of a warp's stage
constexpr int kRedPitch = kTileRows + 4;     // floats between columns of the sums' buffer

template <int F> struct Format;              // elements of K per stage
template <> struct Format<KDA_WEIGHT_BF16> { static constexpr int stage_k = 64, terms = 3; };
template <> struct Format<KDA_WEIGHT_E2M1> { static constexpr int stage_k = 256, terms = 2; };
template <> struct Format<KDA_WEIGHT_INT4> { static constexpr int stage_k = 256, terms = 2; };

// Shared memory of one CTA: ring of stages (reused for the sums), columns, scales of both sides.
template <int F, int NT> struct Layout {
    static constexpr int cols = 8 * NT;
    static constexpr int stages = NT == 1 ? 4 : 3;
    static constexpr int seg = NT <= 2 ? 1024 : 2048 / NT;       // elements of K whose columns are held at once
    static constexpr int seg_chunks = seg / kChunk, seg_units = seg / 32;
    static constexpr int x_pitch = (seg + 32) * 2;               // bytes; 64 past a multiple of 128: no bank conflicts
    static constexpr int s_pitch = seg_units + 4;                // floats
    static constexpr int ring = kWarps * stages * kWarpStage;
    static constexpr int red = cols * kRedPitch * 4;
    static constexpr int x_at = ring > red ? ring : red;
    static constexpr int s_at = x_at + cols * x_pitch;
    static constexpr int xs_at = s_at + (F == KDA_WEIGHT_BF16 ? 0 : kTileRows * s_pitch * 4);
    static constexpr int bytes = xs_at + cols * seg_chunks * 4;
};

// One matrix [rows][K] of weights.
struct Matrix {
    const uint8_t* w;       // codes [rows][K / 2], or bf16 [rows][K]
    const void* scales;     // [rows][K >> (5 + group_shift)]
    int scale_type;         // 0: bytes (exponent + 127), 1: bf16, 2: fp32
    int group_shift;        // log2(group / 32)
};

__device__ __forceinline__ uint32_t smem_addr(const void* p) { return (uint32_t)__cvta_generic_to_shared(p); }
__device__ __forceinline__ void cp_async16_or_zero(uint32_t dst, const void* src, bool valid) {
    const int n = valid ? 16 : 0;
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N> __device__ __forceinline__ void cp_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }
__device__ __forceinline__ uint32_t lds32(uint32_t a) {
    uint32_t v;
    asm volatile("ld.shared.b32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
    return v;
}
__device__ __forceinline__ uint4 lds128(uint32_t a) {
    uint4 v;
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a) : "memory");
    return v;
}

// d = a b + c on 16 x 8 x 16.
template <bool Bf16>
__device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1, const float (&c)[4]) {
    if constexpr (Bf16)
        asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%10, %11, %12, %13};"
            : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(c[0]), "f"(c[1]), "f"(c[2]), "f"(c[3]));
    else
        asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%10, %11, %12, %13};"
            : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(c[0]), "f"(c[1]), "f"(c[2]), "f"(c[3]));
}

// Eight codes as four pairs of fp16.  e2m1: elements (0,1) (2,3) (4,5) (6,7).  int4: a code of four bits put
// into the mantissa of 1024 (or, 16 times itself, of the same) and the offset taken off, which leaves
// elements (0,4) (1,5) (2,6) (3,7); the columns are laid out in that order.
template <int F> __device__ __forceinline__ void widen(uint32_t w, uint32_t (&p)[4]) {
    if constexpr (F == KDA_WEIGHT_E2M1) {
        asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
            "mov.b32 {b0, b1, b2, b3}, %4;\n\t"
            "cvt.rn.f16x2.e2m1x2 %0, b0;\n\tcvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
            "cvt.rn.f16x2.e2m1x2 %2, b2;\n\tcvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
            : "=r"(p[0]), "=r"(p[1]), "=r"(p[2]), "=r"(p[3]) : "r"(w));
    } else {
        const uint32_t h = w >> 8;
        const __half2 one = __half2half2(__ushort_as_half(0x6408));     // 1032
        const __half2 sixteenth = __half2half2(__ushort_as_half(0x2c00));
        const __half2 off = __half2half2(__ushort_as_half(0xd480));     // -72
        auto bits = [](__half2 v) { return *reinterpret_cast<uint32_t*>(&v); };
        auto half = [](uint32_t v) { return *reinterpret_cast<__half2*>(&v); };
        p[0] = bits(__hsub2(half((w & 0x000f000fu) | 0x64006400u), one));
        p[1] = bits(__hfma2(half((w & 0x00f000f0u) | 0x64006400u), sixteenth, off));
        p[2] = bits(__hsub2(half((h & 0x000f000fu) | 0x64006400u), one));
        p[3] = bits(__hfma2(half((h & 0x00f000f0u) | 0x64006400u), sixteenth, off));
    }
}

__device__ __forceinline__ uint32_t pack_half2(float lo, float hi) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
}

// The power of two that brings a magnitude with these fp32 exponent bits to 2^14..2^15 (as far as fp32 has
// one), and its inverse.
__device__ __forceinline__ void run_scale(uint32_t exponent, float& up, float& down) {
    const uint32_t e = 268u - exponent;             // 127 + 14 + 127 - exponent
    const uint32_t b = e > 254u ? 254u : e;
    up = __uint_as_float(b << 23);
    const uint32_t d = 254u - b;
    down = __uint_as_float(d ? d << 23 : 0x00400000u);
}

// A kernel that was launched beside the one in front of it on the stream waits here until that one has ended, and with it
// all before; the one in front lets it begin.  Without such a launch both do nothing.
__device__ __forceinline__ void wait_for_kernel_before() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void let_next_kernel_begin() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

// Launches a kernel in clusters of `ranks` along x, `beside` the kernel in front of it.
template <typename... P, typename... A>
cudaError_t launch_kernel(void (*kernel)(P...), dim3 grid, int threads, int ranks, int smem, bool beside, cudaStream_t s, A&&... args) {
    if (smem > 48 * 1024)
        if (const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem)) return e;
    cudaLaunchAttribute at[2];
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = threads;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cfg.attrs = at;
    if (beside) {
        at[cfg.numAttrs].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        at[cfg.numAttrs++].val.programmaticStreamSerializationAllowed = 1;
    }
    if (ranks > 1) {
        at[cfg.numAttrs].id = cudaLaunchAttributeClusterDimension;
        at[cfg.numAttrs].val.clusterDim.x = ranks;
        at[cfg.numAttrs].val.clusterDim.y = 1;
        at[cfg.numAttrs++].val.clusterDim.z = 1;
    }
    return cudaLaunchKernelEx(&cfg, kernel, std::forward<A>(args)...);
}

// Where the columns come from.  Bf16Rows: column c is row of[c] of a bf16 tensor.  F32Rows: columns
// c * terms .. c * terms + terms - 1 are the parts of fp32 row of[c].
struct Bf16Rows {
    const bf16* x;
    int64_t stride;
    bool wide;  // 16-byte accesses
    static constexpr bool split = false;
};
struct F32Rows {
    const float* x;
    int64_t stride;
    static constexpr bool split = true;
};

// 16 bytes of a column (eight elements from k, a multiple of 8) to their places in shared memory.
template <int F>
__device__ __forceinline__ void put8(uint8_t* col, int k, const uint32_t (&v)[4]) {
    if constexpr (F == KDA_WEIGHT_E2M1) {
        *reinterpret_cast<uint4*>(col + 2 * k) = make_uint4(v[0], v[1], v[2], v[3]);
    } else if constexpr (F == KDA_WEIGHT_INT4) {
        *reinterpret_cast<uint4*>(col + 2 * k) = make_uint4(__byte_perm(v[0], v[2], 0x5410), __byte_perm(v[0], v[2], 0x7632),
                                                            __byte_perm(v[1], v[3], 0x5410), __byte_perm(v[1], v[3], 0x7632));
    } else {  // word t of the four accesses of 32 elements next to each other: the order the lanes read them in
        uint32_t* p = reinterpret_cast<uint32_t*>(col + 2 * (k & ~31)) + ((k >> 3) & 3);
        p[0] = v[0];
        p[4] = v[1];
        p[8] = v[2];
        p[12] = v[3];
    }
}

// Columns [0, n) of K in [k0, k0 + seg) (zeros from k1 and past the last column) into shared memory.
template <int F, int NT, typename Src>
__device__ __forceinline__ void stage_columns(uint8_t* smem, const Src& src, const int* of, int n, int k0, int k1) {
    using L = Layout<F, NT>;
    constexpr int kTerms = Src::split ? Format<F>::terms : 1;
    constexpr int kBatch = Src::split ? 2 : 4;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    float* xs = reinterpret_cast<float*>(smem + L::xs_at);
    const int chunks = min(L::seg_chunks, (k1 - k0 + kChunk - 1) / kChunk);
    const int items = n * chunks;
    for (int it0 = warp; it0 < items; it0 += kWarps * kBatch) {
        uint32_t v[kBatch][Src::split ? 8 : 4];
#pragma unroll
        for (int b = 0; b < kBatch; ++b) {
            const int it = it0 + b * kWarps, c = it / chunks, k = k0 + (it - c * chunks) * kChunk + lane * 8;
#pragma unroll
            for (int i = 0; i < (Src::split ? 8 : 4); ++i) v[b][i] = 0;
            if (it < items && k < k1) {
                if constexpr (Src::split) {
                    const float4* p = reinterpret_cast<const float4*>(src.x + (int64_t)of[c] * src.stride + k);
                    const float4 lo = p[0], hi = p[1];
                    v[b][0] = __float_as_uint(lo.x), v[b][1] = __float_as_uint(lo.y), v[b][2] = __float_as_uint(lo.z);
                    v[b][3] = __float_as_uint(lo.w), v[b][4] = __float_as_uint(hi.x), v[b][5] = __float_as_uint(hi.y);
                    v[b][6] = __float_as_uint(hi.z), v[b][7] = __float_as_uint(hi.w);
                } else {
                    const bf16* p = src.x + (int64_t)of[c] * src.stride + k;
                    if (src.wide) {
                        const uint4 q = *reinterpret_cast<const uint4*>(p);
                        v[b][0] = q.x, v[b][1] = q.y, v[b][2] = q.z, v[b][3] = q.w;
                    } else {
                        const unsigned short* h = reinterpret_cast<const unsigned short*>(p);
#pragma unroll
                        for (int i = 0; i < 4; ++i) v[b][i] = h[2 * i] | ((uint32_t)h[2 * i + 1] << 16);
                    }
                }
            }
        }
#pragma unroll
        for (int b = 0; b < kBatch; ++b) {
            const int it = it0 + b * kWarps, c = it / chunks, ch = it - c * chunks;
            if (it >= items) break;
            const int k = ch * kChunk + lane * 8;
            uint8_t* col = smem + L::x_at + c * kTerms * L::x_pitch;
            if constexpr (F == KDA_WEIGHT_BF16) {
                if constexpr (!Src::split) {
                    put8<F>(col, k, v[b]);
                } else {
                    float r[8];
#pragma unroll
                    for (int i = 0; i < 8; ++i) r[i] = __uint_as_float(v[b][i]);
#pragma unroll
                    for (int t = 0; t < kTerms; ++t) {
                        uint32_t o[4];
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const bf16 a = __float2bfloat16_rn(r[2 * i]), c2 = __float2bfloat16_rn(r[2 * i + 1]);
                            o[i] = (uint32_t)__bfloat16_as_ushort(a) | ((uint32_t)__bfloat16_as_ushort(c2) << 16);
                            const float fa = __bfloat162float(a), fb = __bfloat162float(c2);
                            r[2 * i] = isinf(fa) ? 0.f : r[2 * i] - fa;
                            r[2 * i + 1] = isinf(fb) ? 0.f : r[2 * i + 1] - fb;
                        }
                        put8<F>(col + t * L::x_pitch, k, o);
                    }
                }
            } else {
                uint32_t top = 0;
                if constexpr (Src::split) {
#pragma unroll
                    for (int i = 0; i < 8; ++i) top = max(top, v[b][i] & 0x7fffffffu);
                } else {
#pragma unroll
                    for (int i = 0; i < 4; ++i) top = __vmaxu2(top, v[b][i] & 0x7fff7fffu);
                    top = max(top << 16, top & 0xffff0000u);
                }
                top = __reduce_max_sync(0xffffffffu, top);
                float up, down;
                run_scale(top >> 23, up, down);
                float r[8];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    if constexpr (Src::split) {
                        r[2 * i] = __uint_as_float(v[b][2 * i]) * up;
                        r[2 * i + 1] = __uint_as_float(v[b][2 * i + 1]) * up;
                    } else {
                        r[2 * i] = __uint_as_float(v[b][i] << 16) * up;
                        r[2 * i + 1] = __uint_as_float(v[b][i] & 0xffff0000u) * up;
                    }
                }
#pragma unroll
                for (int t = 0; t < kTerms; ++t) {
                    uint32_t o[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        o[i] = pack_half2(r[2 * i], r[2 * i + 1]);
                        if constexpr (kTerms > 1) {
                            const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&o[i]));
                            r[2 * i] = isinf(f.x) ? 0.f : r[2 * i] - f.x;
                            r[2 * i + 1] = isinf(f.y) ? 0.f : r[2 * i + 1] - f.y;
                        }
                    }
                    put8<F>(col + t * L::x_pitch, k, o);
                    if (lane == 0) xs[(c * kTerms + t) * L::seg_chunks + ch] = down;
                }
            }
        }
    }
}

// Zeros for the columns that hold no token: what multiplies them is never read, but must not trap or turn up as NaN in
// other columns' runs.
template <int F, int NT> __device__ __forceinline__ void clear_columns(uint8_t* smem, int used) {
    using L = Layout<F, NT>;
    float* xs = reinterpret_cast<float*>(smem + L::xs_at);
    uint4* x = reinterpret_cast<uint4*>(smem + L::x_at + used * L::x_pitch);
    for (int i = threadIdx.x; i < (L::cols - used) * (L::x_pitch / 16); i += kThreads) x[i] = make_uint4(0, 0, 0, 0);
    if constexpr (F != KDA_WEIGHT_BF16)
        for (int i = used * L::seg_chunks + threadIdx.x; i < L::cols * L::seg_chunks; i += kThreads) xs[i] = 0.f;
}

// Scales of the tile's rows for K in [k0, k0 + seg), one fp32 per row and 32 elements (zeros from k1).
// row_of(r): the tile's row r as a row of the matrix.
template <int F, int NT, typename RowOf>
__device__ __forceinline__ void stage_scales(uint8_t* smem, const Matrix& m, int K, const RowOf& row_of, int k0, int k1) {
    using L = Layout<F, NT>;
    float* sc = reinterpret_cast<float*>(smem + L::s_at);
    const int64_t per_row = K >> (5 + m.group_shift);
    const int u0 = k0 >> 5, units = min(L::seg_units, (k1 - k0) >> 5);
    // two threads per row, each half of the row's units: four at a time
    const int r = threadIdx.x >> 1;
    const int64_t row = row_of(r) * per_row;
    float* dst = sc + r * L::s_pitch;
    const bool quads = m.scale_type == 0 && m.group_shift == 0 && (per_row & 3) == 0 &&
                       (reinterpret_cast<uintptr_t>(m.scales) & 3) == 0 && (units & 3) == 0;
    if (quads) {
        const uint32_t* p = reinterpret_cast<const uint32_t*>(static_cast<const uint8_t*>(m.scales) + row + u0);
#pragma unroll 4
        for (int q = threadIdx.x & 1; q < L::seg_units / 4; q += 2) {
            const uint32_t b = q * 4 < units ? p[q] : 0;
            *reinterpret_cast<float4*>(dst + 4 * q) =
                make_float4(__uint_as_float((b & 0xffu) << 23), __uint_as_float((b & 0xff00u) << 15),
                            __uint_as_float((b & 0xff0000u) << 7), __uint_as_float((b >> 24) << 23));
        }
        return;
    }
#pragma unroll 4
    for (int u = threadIdx.x & 1; u < L::seg_units; u += 2) {
        float v = 0.f;
        if (u < units) {
            const int64_t at = row + ((u0 + u) >> m.group_shift);
            if (m.scale_type == 0)
                v = __uint_as_float((uint32_t)static_cast<const uint8_t*>(m.scales)[at] << 23);
            else if (m.scale_type == 1)
                v = __bfloat162float(static_cast<const bf16*>(m.scales)[at]);
            else
                v = static_cast<const float*>(m.scales)[at];
        }
        dst[u] = v;
    }
}

// acc[n][.] += the tile's 128 rows times up to 8 NT columns over K in [k0, k1) (k0 a multiple of 256): a lane
// of a warp holds rows g and g + 8 of its 16 and columns 8 n + 2 t, + 1.
template <int F, int NT, typename Src, typename RowOf>
__device__ __forceinline__ void product(uint8_t* smem, const Matrix& m, int K, const RowOf& row_of, const Src& src,
                                        const int* of, int n, int k0, int k1, float (&acc)[NT][4]) {
    using L = Layout<F, NT>;
    constexpr int kStageK = Format<F>::stage_k;
    constexpr bool kBf16 = F == KDA_WEIGHT_BF16;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
#pragma unroll
    for (int i = 0; i < NT; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = 0.f;
    if (k1 <= k0) return;  // the whole CTA: more ranks than runs of 256

    const int64_t pitch = kBf16 ? (int64_t)K * 2 : (int64_t)K / 2;
    const int slice = kBf16 ? (k1 - k0) * 2 : (k1 - k0) / 2;  // bytes of a row
    const int total = (slice + kRowStage - 1) / kRowStage;
    const uint32_t ring = smem_addr(smem) + warp * L::stages * kWarpStage;
    const int piece = lane & 7, r0 = lane >> 3;
    const uint8_t* from[4];
    uint32_t to[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int r = r0 + 4 * i;
        from[i] = m.w + row_of(16 * warp + r) * pitch + (kBf16 ? (int64_t)k0 * 2 : (int64_t)k0 / 2) + piece * 16;
        to[i] = ring + r * kRowStage + ((piece ^ (r & 7)) << 4);
    }
    auto issue = [&](int c) {
        if (c < total) {
            const bool in = c * kRowStage + piece * 16 < slice;
            const uint32_t slot = (uint32_t)(c % L::stages) * kWarpStage;
#pragma unroll
            for (int i = 0; i < 4; ++i) cp_async16_or_zero(to[i] + slot, in ? from[i] + (int64_t)c * kRowStage : m.w, in);
        }
        cp_commit();
    };
#pragma unroll
    for (int c = 0; c < L::stages - 1; ++c) issue(c);

    const uint32_t col = smem_addr(smem) + L::x_at + g * L::x_pitch + t * 16;
    const float* sc0 = reinterpret_cast<const float*>(smem + L::s_at) + (16 * warp + g) * L::s_pitch;
    const float* sc1 = sc0 + 8 * L::s_pitch;
    const float* xs = reinterpret_cast<const float*>(smem + L::xs_at);
    const float zero[4] = {0.f, 0.f, 0.f, 0.f};
    clear_columns<F, NT>(smem, n * (Src::split ? Format<F>::terms : 1));
    int c = 0;
    for (int seg = k0; seg < k1; seg += L::seg) {
        if (seg != k0) __syncthreads();  // every warp is done with the last columns
        if constexpr (!kBf16) stage_scales<F, NT>(smem, m, K, row_of, seg, k1);
        stage_columns<F, NT>(smem, src, of, n, seg, k1);
        __syncthreads();
        const int runs = (min(k1 - seg, L::seg) + kStageK - 1) / kStageK;
        for (int run = 0; run < runs; ++run, ++c) {
            cp_wait<L::stages - 2>();
            __syncwarp();
            issue(c + L::stages - 1);
            const uint32_t wrow = ring + (uint32_t)(c % L::stages) * kWarpStage + g * kRowStage + t * 4;
            if constexpr (kBf16) {
                // a stage's sum starts from zero and is added in fp32: the matrix instructions drop digits below the
                // accumulator's last one, which over a long chain takes 5 of its 24 bits
                float part[NT][4];
#pragma unroll
                for (int i = 0; i < NT; ++i)
#pragma unroll
                    for (int j = 0; j < 4; ++j) part[i][j] = 0.f;
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    uint32_t w[4][2];
#pragma unroll
                    for (int p = 0; p < 4; ++p) {
                        const uint32_t at = wrow + (((4 * h + p) ^ g) << 4);
                        w[p][0] = lds32(at);
                        w[p][1] = lds32(at + 8 * kRowStage);
                    }
#pragma unroll
                    for (int i = 0; i < NT; ++i) {
                        const uint4 x = lds128(col + i * 8 * L::x_pitch + (run * kStageK + 32 * h) * 2);
                        const uint32_t a0[4] = {w[0][0], w[0][1], w[1][0], w[1][1]};
                        const uint32_t a1[4] = {w[2][0], w[2][1], w[3][0], w[3][1]};
                        mma<true>(part[i], a0, x.x, x.y, part[i]);
                        mma<true>(part[i], a1, x.z, x.w, part[i]);
                    }
                }
#pragma unroll
                for (int i = 0; i < NT; ++i)
#pragma unroll
                    for (int j = 0; j < 4; ++j) acc[i][j] += part[i][j];
            } else {
                float part[NT][4];
#pragma unroll
                for (int i = 0; i < NT; ++i)
#pragma unroll
                    for (int j = 0; j < 4; ++j) part[i][j] = 0.f;
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const float4 s0 = *reinterpret_cast<const float4*>(sc0 + run * 8 + 4 * h);
                    const float4 s1 = *reinterpret_cast<const float4*>(sc1 + run * 8 + 4 * h);
                    const float f0[4] = {s0.x, s0.y, s0.z, s0.w}, f1[4] = {s1.x, s1.y, s1.z, s1.w};
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        const int j = 4 * h + q;
                        const uint32_t at = wrow + ((j ^ g) << 4);
                        uint32_t lo[4], hi[4];
                        widen<F>(lds32(at), lo);
                        widen<F>(lds32(at + 8 * kRowStage), hi);
                        const uint32_t a0[4] = {lo[0], hi[0], lo[1], hi[1]}, a1[4] = {lo[2], hi[2], lo[3], hi[3]};
#pragma unroll
                        for (int i = 0; i < NT; ++i) {
                            const uint4 x = lds128(col + i * 8 * L::x_pitch + (run * kChunk + 32 * j) * 2);
                            float d[4];
                            mma<false>(d, a0, x.x, x.y, zero);
                            mma<false>(d, a1, x.z, x.w, d);
                            part[i][0] = fmaf(f0[q], d[0], part[i][0]);
                            part[i][1] = fmaf(f0[q], d[1], part[i][1]);
                            part[i][2] = fmaf(f1[q], d[2], part[i][2]);
                            part[i][3] = fmaf(f1[q], d[3], part[i][3]);
                        }
                    }
                }
#pragma unroll
                for (int i = 0; i < NT; ++i) {
                    const float x0 = xs[(8 * i + 2 * t) * L::seg_chunks + run], x1 = xs[(8 * i + 2 * t + 1) * L::seg_chunks + run];
                    acc[i][0] = fmaf(x0, part[i][0], acc[i][0]);
                    acc[i][1] = fmaf(x1, part[i][1], acc[i][1]);
                    acc[i][2] = fmaf(x0, part[i][2], acc[i][2]);
                    acc[i][3] = fmaf(x1, part[i][3], acc[i][3]);
                }
            }
        }
    }
    cp_wait<0>();
}

// The tile's sums from the lanes to the buffer [column][128 rows] in shared memory (over the ring), visible to
// the whole cluster when it returns.
template <int F, int NT> __device__ __forceinline__ float* gather(uint8_t* smem, const float (&acc)[NT][4], int ranks) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    float* red = reinterpret_cast<float*>(smem);
    __syncthreads();  // every warp is done with the ring
#pragma unroll
    for (int i = 0; i < NT; ++i) {
        float* p = red + (8 * i + 2 * t) * kRedPitch + 16 * warp + g;
        p[0] = acc[i][0];
        p[kRedPitch] = acc[i][1];
        p[8] = acc[i][2];
        p[kRedPitch + 8] = acc[i][3];
    }
    if (ranks > 1) cooperative_groups::this_cluster().sync(); else __syncthreads();
    return red;
}

// One element of the joined tile: column c (or the terms of row c) and tile row r, ranks added in their order.
template <int Terms> __device__ __forceinline__ float joined(float* red, int ranks, int c, int r) {
    float v = 0.f;
    for (int rank = 0; rank < ranks; ++rank) {
        const float* p = ranks > 1 ? cooperative_groups::this_cluster().map_shared_rank(red, rank) : red;
        float one = p[c * Terms * kRedPitch + r];
#pragma unroll
        for (int t = 1; t < Terms; ++t) one += p[(c * Terms + t) * kRedPitch + r];
        v = rank ? v + one : one;
    }
    return v;
}

// Before the buffer is written again, or the CTA ends: nobody reads it any more.
__device__ __forceinline__ void release(int ranks) {
    if (ranks > 1) cooperative_groups::this_cluster().sync(); else __syncthreads();
}

// The part of K that this rank takes, in whole runs of 256.
__device__ __forceinline__ void slice_of(int K, int rank, int ranks, int& k0, int& k1) {
    const int runs = (K + kChunk - 1) / kChunk;
    k0 = (int)((int64_t)runs * rank / ranks) * kChunk;
    k1 = min(K, (int)((int64_t)runs * (rank + 1) / ranks) * kChunk);
}

// CTAs of a cluster that share a tile's K: the number with the shortest run of rounds of CTAs, where a CTA's time is
// its runs of 256 and about four more to start and to join.
inline int cluster_ranks(int64_t tiles, int K) {
    const int runs = (K + kChunk - 1) / kChunk, at_once = 2 * 152;
    int best = 1;
    double least = 1e300;
    for (int r = 1; r <= 8 && r <= runs; r *= 2) {
        const int64_t ctas = tiles * r;
        const double rounds = ctas <= at_once ? 1.0 : (double)ctas / at_once + 0.5;
        const double t = rounds * ((double)runs / r + 4.0);
        if (t < least) least = t, best = r;
    }
    return best;
}

}  // namespace few
}  // namespace kda
