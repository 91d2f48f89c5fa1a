// kda_few.cuh -- products of a matrix of integer codes in 4 bits with a few columns (tokens): what the 4-bit projections
// (kda_gemm4.cu) and the experts (kda_moe.cu) share for weights (code - 8) * scale, one scale per 32, 64 or 128 weights.
//
// Bound by the codes' bytes and by the instructions that take them apart.  A scale of any value cannot go to the
// block-scaled tensor cores, so codes become fp16 operands of mma.sync (m16n8k16, fp32 accumulation: its narrow side of 8
// fits a few tokens) by a shift and a mask: four bits in a half's mantissa are the subnormal code 2^-20.  The 8 to be taken
// off is not taken off the codes: a group's sum starts from -8 times the sum of the column's elements in it.  (Codes as
// 1024 + code, 1032 taken off in registers, were 16 instructions more per 512 weights.)  A group's sum is multiplied by
// the weights' scale in fp32 when it is added up: scales are never rounded.
//
// The instruction lines products up by their operands' exponents, which for a subnormal is that of 2^-14 whatever its
// leading zeros, and drops what lies too far below the largest.  Codes lie in mantissa bits 4 to 7, which leaves 1.2e-7 of
// a product over 2,048 elements.  In bits 0 to 3 for every other element (no shift for three of four) it was
// 5e-7, and 4e-6 to 7e-6 for experts, whose hidden values spread over more exponents; 160,000 x 7,168 codes and 16 tokens
// took 178 us against 185.
//
// Columns are prepared by a kernel in front (k_few_halves): each run of 128 elements is brought to 2^14..2^15 by a
// power of two, which is exact for a bf16 element down to 2^-31 of its run's largest and off by at most 2^-39 of the largest
// below that, less than an fp32 sum would keep; fp32 values are two columns, value and remainder.  The power's
// inverse is multiplied in at the end of a run.
//
// A CTA has 8 or 12 warps.  A warp takes 32 rows, two tiles of an instruction, so that each operand of the columns is read from
// shared memory once for both and their chains of instructions overlap (16 warps of 16 rows each: 12 % longer for 160,000
// x 7,168 codes and 16 tokens).  Its codes and scales go through cp.async into a ring of its own
// (32 rows x 256 elements a stage), no barrier among warps.  All columns of a segment of K are in shared memory for all
// warps, the next segment's on their way meanwhile: one barrier per segment.  `ks` warps share 32 rows along K where there
// are few rows.
#pragma once

#include <cooperative_groups.h>
#include <cuda_fp16.h>

#include <utility>

#include "kda_internal.cuh"

namespace kda {
namespace few {

constexpr int kTileRows = 128;               // rows of a tile on the tensor cores (kda_few_tc.cuh)
constexpr int kRedPitch = kTileRows + 4;     // floats between columns of its sums

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

constexpr int kRows = 32;                    // of a warp
constexpr int kStageK = 256;                 // elements of a row per stage
constexpr int kRun = 128;                    // elements of a column under one power of two
constexpr int kWarpStage = kRows * kStageK / 2; // bytes of codes in a warp's stage
constexpr int kStages = 3;

// A CTA of W warps for 8 NT columns, GS groups in a stage and SB bytes of a scale.
template <int W_, int NT_, int GS_, int SB_> struct Layout {
    static constexpr int W = W_, NT = NT_, GS = GS_, SB = SB_, threads = 32 * W;
    static constexpr int cols = 8 * NT, scale_row = GS * SB;     // bytes of a row's scales in a stage
    static constexpr int seg = 2048 / NT, seg_stages = seg / kStageK, seg_runs = seg / kRun;
    static constexpr int most_ks = seg_stages / 2;               // a warp has two stages of a segment at least
    static constexpr int x_pitch = (seg + 32) * 2;               // bytes; 64 past a multiple of 128: no bank conflicts
    static constexpr int scales_at = W * kStages * kWarpStage;
    static constexpr int x_at = scales_at + W * kStages * kRows * scale_row;
    static constexpr int f_at = x_at + 2 * cols * x_pitch;       // [2][cols][seg_runs]
    static constexpr int most_groups = seg / 32;                 // of a segment: sums [2][groups][cols]
    static constexpr int sums_at = f_at + 2 * cols * seg_runs * 4;
    static constexpr int bytes = sums_at + 2 * most_groups * cols * 4;
    static_assert(most_ks < 2 || W * kRows * cols * 4 <= cols * x_pitch, "sums of warps that share rows fit over a segment's columns");
    static_assert(bytes <= 227 * 1024, "shared memory of an SM");
};

struct Weights {  // of one matrix [rows][K]
    const uint8_t* codes;
    const uint8_t* scales;
};
struct Columns {  // laid out by k_few_halves
    const __half* x;      // [.][K]
    const float* factor;  // [.][runs of 128]: what a sum is to be multiplied by
    const float* sums;    // [.][groups]: -8 2^-20 times the sum of a group's elements
};

__device__ __forceinline__ uint32_t smem_addr(const void* p) { return (uint32_t)__cvta_generic_to_shared(p); }
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, int n) {  // zeros behind the first n bytes
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
}
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async8(uint32_t dst, const void* src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async4(uint32_t dst, const void* src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N> __device__ __forceinline__ void cp_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }
// d = a b + c on 16 x 8 x 16.
__device__ __forceinline__ void mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1, const float (&c)[4]) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%10, %11, %12, %13};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(c[0]), "f"(c[1]), "f"(c[2]), "f"(c[3]));
}

// Eight codes as four pairs of fp16, code 2^-20: elements (0,4), (1,5), (2,6), (3,7).  The columns are laid out in that order.
__device__ __forceinline__ void part(uint32_t w, uint32_t (&p)[4]) {
    p[0] = w << 4 & 0x00f000f0u;
    p[1] = w & 0x00f000f0u;
    p[2] = w >> 4 & 0x00f000f0u;
    p[3] = w >> 8 & 0x00f000f0u;
}

__device__ __forceinline__ uint32_t pack_half2(float lo, float hi) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
}

// The power of two that brings a magnitude with these fp32 exponent bits to 2^14..2^15 (as far as fp32 has
// one), and what sums of subnormal codes are to be multiplied by: its inverse times 2^20.  Magnitudes from 2^122 on, for which
// fp32 has none, get NaN.
__device__ __forceinline__ void run_scale(uint32_t exponent, float& up, float& down) {
    const uint32_t e = 268u - exponent;             // 127 + 14 + 127 - exponent
    const uint32_t b = e > 254u ? 254u : e;
    up = __uint_as_float(b << 23);
    const uint32_t d = 254u - b + 20u;
    down = d < 255u ? __uint_as_float(d << 23) : NAN;
}

// Where the columns of `n` rows of K elements lie in a buffer, and what they take.
inline Columns columns_at(void* buffer, int64_t n, int64_t K) {
    __half* x = static_cast<__half*>(buffer);
    float* factor = reinterpret_cast<float*>(x + n * K);
    return Columns{x, factor, factor + n * ((K + kRun - 1) / kRun)};
}
inline size_t columns_bytes(int64_t n, int64_t K, int group) {
    return (size_t)n * K * 2 + (size_t)n * ((K + kRun - 1) / kRun) * 4 + (size_t)n * (K / group) * 4;
}
// The columns of bf16 rows [rows][K] (K a multiple of the group).
cudaError_t launch_halves(const bf16* x, int64_t xs, bool wide, int rows, int K, int group, const Columns& columns, cudaStream_t s);

constexpr float kSumOf = -8.f * 0x1p-20f;

// One product by itself, for a sum that came out as NaN or infinite: a row of x with an infinity or values that no factor is for, or
// scales from 2^123 on (a run's sum, before its factor, is up to 2^5 of them).  An eighth
// of the weight times x, so that neither a scale nor an x next to the end of fp32 overflows where the product does not.
static __device__ __noinline__ float direct(const uint8_t* codes, const uint8_t* scales, int scale_bytes, int group, const bf16* x, int K) {
    float sum = 0.f;
    for (int g = 0; g < K / group; ++g) {
        const float s = scale_bytes == 2 ? to_f(reinterpret_cast<const bf16*>(scales)[g]) : reinterpret_cast<const float*>(scales)[g];
        for (int i = g * group; i < (g + 1) * group; ++i) {
            const float eighth = 0.125f * ((int)(codes[i >> 1] >> (4 * (i & 1)) & 15u) - 8);
            sum = fmaf(eighth * s, to_f(x[i]), sum);
        }
    }
    return 8.f * sum;
}

// The same with a hidden value's two columns (value and remainder, laid out by k_moe_in): NaN where a run has no factor.
static __device__ __noinline__ float direct_columns(const uint8_t* codes, const uint8_t* scales, int scale_bytes, int group, const __half* hi,
                                                    const __half* lo, const float* factor, int K) {
    float sum = 0.f;
    for (int r = 0; r * kRun < K; ++r)
        if (isnan(factor[r])) return NAN;
    for (int k = 0; k < K; ++k) {
        const float s = scale_bytes == 2 ? to_f(reinterpret_cast<const bf16*>(scales)[k / group]) : reinterpret_cast<const float*>(scales)[k / group];
        const float eighth = 0.125f * ((int)(codes[k >> 1] >> (4 * (k & 1)) & 15u) - 8);
        const int at = (k & ~7) + 2 * (k & 3) + (k >> 2 & 1);
        const float x = (__half2float(hi[at]) + __half2float(lo[at])) * (factor[k / kRun] * 0x1p-20f);
        sum = fmaf(eighth * s, x, sum);
    }
    return 8.f * sum;
}

// The sums of a CTA.  row_of(pass, tile, r): the matrix's row of row r of one of the W / ks tiles of 32 rows that the CTA
// takes in a pass, or -1 for a tile that does not exist; column c is row of[c] of the columns' tensor, c < n.  After each
// pass the warps call done(pass, acc) with a lane's sums: acc[u] holds rows 16 u + g and + 8 of the warp's tile (warp / ks),
// columns 8 i + 2 t, + 1; where ks warps share a tile the first of them holds the sums.
template <typename L, typename RowOf, typename Done>
__device__ __forceinline__ void products(uint8_t* smem, const Weights& w, const Columns& x, int K, const int* of, int n, int ks, int passes,
                                         const RowOf& row_of, const Done& done) {
    constexpr int NT = L::NT, GS = L::GS, SB = L::SB, kThreads = L::threads, kScaleRow = L::scale_row;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const int tile = warp / ks, slot = warp - tile * ks;
    const int stages = (K + kStageK - 1) / kStageK, segs = (K + L::seg - 1) / L::seg, own = L::seg_stages / ks, runs = (K + kRun - 1) / kRun;
    const int row_scales = K / (kStageK / GS);
    const uint32_t ring = smem_addr(smem) + warp * kStages * kWarpStage;
    const uint32_t sring = smem_addr(smem) + L::scales_at + warp * kStages * kRows * kScaleRow;
    const int piece = lane & 7, r0 = lane >> 3;
    constexpr int kStageScales = GS * SB, kUnit = kStageScales < 16 ? kStageScales : 16;  // bytes of a row's scales, and of a copy
    const bool whole = ((uint64_t)(row_scales * SB) | reinterpret_cast<uint64_t>(w.scales)) % kUnit == 0;

    // columns of segment q (counted over the passes) into buffer q & 1, 8 elements at a time
    constexpr int kPieces = L::seg / 8;
    const auto load_columns = [&](int q) {
        const int s = q % segs;
        const uint32_t to = smem_addr(smem) + L::x_at + (q & 1) * L::cols * L::x_pitch;
#pragma unroll 4
        for (int i = threadIdx.x; i < L::cols * kPieces; i += kThreads) {
            const int c = i / kPieces, k = i % kPieces * 8;
            const bool in = c < n && s * L::seg + k < K;
            cp_async16(to + c * L::x_pitch + k * 2, in ? x.x + (int64_t)of[c] * K + s * L::seg + k : x.x, in ? 16 : 0);
        }
        if (threadIdx.x < L::cols * L::seg_runs) {
            float* f = reinterpret_cast<float*>(smem + L::f_at) + (q & 1) * L::cols * L::seg_runs + threadIdx.x;
            const int c = threadIdx.x / L::seg_runs, r = s * L::seg_runs + threadIdx.x % L::seg_runs;
            if (c < n && r < runs)
                cp_async4(smem_addr(f), x.factor + (int64_t)of[c] * runs + r);
            else
                *f = 0.f;
        }
        constexpr int kGroups = L::seg_stages * GS;  // of a segment
        for (int i = threadIdx.x; i < kGroups * L::cols; i += kThreads) {
            const int c = i / kGroups, j = i % kGroups, at = s * kGroups + j;
            float* f = reinterpret_cast<float*>(smem + L::sums_at) + (q & 1) * L::most_groups * L::cols + j * L::cols + c;
            if (c < n && at < row_scales)
                cp_async4(smem_addr(f), x.sums + (int64_t)of[c] * row_scales + at);
            else
                *f = 0.f;
        }
    };

    // this warp's stages, counted over passes, segments and its share of a segment's stages
    const uint8_t *row = nullptr, *srow = nullptr;  // of this lane's first piece and of its row's scales, at K = 0
    bool inside = false;                            // all 32 rows are rows of their own, one after another
    int ipass = -1;                                 // the pass that these belong to
    const int64_t every4 = (int64_t)K * 2;          // bytes between rows r and r + 4
    const uint32_t to_even = ring + r0 * 128 + ((piece ^ r0) << 4), to_odd = ring + (r0 + 4) * 128 + ((piece ^ (r0 + 4)) << 4);
    const uint32_t to_scales = sring + lane * kScaleRow;
    const auto issue = [&](int pass, int st, int buffer) {
        if (pass >= passes || st >= stages) return;
        if (pass != ipass) {
            ipass = pass;
            const int64_t r = row_of(pass, tile, r0), s = row_of(pass, tile, lane);
            row = r < 0 ? nullptr : w.codes + r * (K / 2) + piece * 16;
            srow = r < 0 ? nullptr : w.scales + s * row_scales * SB;
            inside = r >= 0 && row_of(pass, tile, kRows - 1) == row_of(pass, tile, 0) + kRows - 1;
        }
        if (!row) return;
        const uint32_t off = buffer * kWarpStage;
        const bool full = (st + 1) * kStageK <= K;
        if (inside && full) {
            const uint8_t* p = row + st * 128;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                cp_async16((i & 1 ? to_odd : to_even) + off + (i >> 1) * 1024, p);
                p += every4;
            }
        } else {
            const int left = K / 2 - st * 128 - piece * 16;  // bytes of a row from here
#pragma unroll 1
            for (int i = 0; i < 8; ++i) {
                const uint8_t* p = w.codes + row_of(pass, tile, r0 + 4 * i) * (K / 2);
                cp_async16((i & 1 ? to_odd : to_even) + off + (i >> 1) * 1024, left > 0 ? p + st * 128 + piece * 16 : p, left > 0 ? 16 : 0);
            }
        }
        // a row's scales per lane
        const uint32_t sto = to_scales + buffer * kRows * kScaleRow;
        const uint8_t* from = srow + st * kStageScales;
        if (whole && full) {
            if constexpr (kUnit == 4) cp_async4(sto, from);
            else if constexpr (kUnit == 8) cp_async8(sto, from);
            else cp_async16(sto, from);
            if constexpr (kStageScales == 32) cp_async16(sto + 16, from + 16);
        } else {
            const int have = min(GS, row_scales - st * GS) * SB;
            for (int b = 0; b < kStageScales; b += 2)  // zeros for groups behind K
                asm volatile("st.shared.b16 [%0], %1;" ::"r"(sto + b), "h"(b < have ? *reinterpret_cast<const unsigned short*>(from + b) : (unsigned short)0) : "memory");
        }
    };
    int l_pass = 0, l_seg = 0, l_i = 0, l_buffer = 0;  // the next stage to issue
    const auto advance = [&]() {
        issue(l_pass, l_seg * L::seg_stages + l_i * ks + slot, l_buffer);
        if (++l_buffer == kStages) l_buffer = 0;
        if (++l_i == own) {
            l_i = 0;
            if (++l_seg == segs) l_seg = 0, ++l_pass;
        }
    };

    load_columns(0);
    advance();
    cp_commit();
    advance();
    cp_commit();
    int buffer = 0;
    for (int pass = 0; pass < passes; ++pass) {
        float acc[2][NT][4];
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
            for (int i = 0; i < NT; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) acc[u][i][j] = 0.f;
        const bool active = row_of(pass, tile, 0) >= 0;
        for (int s = 0; s < segs; ++s) {
            const int q = pass * segs + s;
            for (int i = 0; i < own; ++i) {
                cp_wait<1>();
                if (i == 0) {
                    __syncthreads();  // everyone's columns are there, and nobody reads the other buffer any more
                    if (q + 1 < passes * segs) load_columns(q + 1);
                } else {
                    __syncwarp();
                }
                advance();
                cp_commit();
                const int at_stage = i * ks + slot;  // in the segment
                if (active && s * L::seg_stages + at_stage < stages) {
                    const uint8_t* col = smem + L::x_at + (q & 1) * L::cols * L::x_pitch + g * L::x_pitch + t * 16 + at_stage * kStageK * 2;
                    const uint32_t wrow = (warp * kStages * kWarpStage + buffer * kWarpStage + g * 128 + t * 4) ^ (g << 4);
                    const uint8_t* srow_at = smem + L::scales_at + (warp * kStages * kRows + buffer * kRows + g) * kScaleRow;
                    const float* f = reinterpret_cast<const float*>(smem + L::f_at) + (q & 1) * L::cols * L::seg_runs + 2 * t * L::seg_runs + at_stage * 2;
                    const float* sum = reinterpret_cast<const float*>(smem + L::sums_at) + (q & 1) * L::most_groups * L::cols + at_stage * GS * L::cols + 2 * t;
#pragma unroll 1
                    for (int h = 0; h < 2; ++h) {  // runs of 128; both unrolled are too much code for the instruction cache
                        constexpr int kHalf = GS / 2, kUnits = 4 / kHalf;  // groups of a run, units of 32 of a group
                        float run[2][NT][4];
#pragma unroll
                        for (int j = 0; j < kHalf; ++j) {
                            float sc[4];  // of rows g, g + 8, g + 16, g + 24
#pragma unroll
                            for (int r = 0; r < 4; ++r) {
                                const uint8_t* p = srow_at + 8 * r * kScaleRow + (h * kHalf + j) * SB;
                                sc[r] = SB == 2 ? __uint_as_float((uint32_t)*reinterpret_cast<const unsigned short*>(p) << 16) : *reinterpret_cast<const float*>(p);
                            }
                            float d[2][NT][4];
#pragma unroll
                            for (int c = 0; c < NT; ++c) {
                                const float2 v = *reinterpret_cast<const float2*>(sum + (h * kHalf + j) * L::cols + 8 * c);
#pragma unroll
                                for (int u = 0; u < 2; ++u) d[u][c][0] = d[u][c][2] = v.x, d[u][c][1] = d[u][c][3] = v.y;
                            }
#pragma unroll
                            for (int k = 0; k < kUnits; ++k) {
                                const int unit = h * 4 + j * kUnits + k;
                                const uint8_t* at = smem + (wrow ^ (unit << 4));
                                uint32_t a[4][4];
#pragma unroll
                                for (int r = 0; r < 4; ++r) part(*reinterpret_cast<const uint32_t*>(at + r * 1024), a[r]);
#pragma unroll
                                for (int c = 0; c < NT; ++c) {
                                    const uint4 b = *reinterpret_cast<const uint4*>(col + c * 8 * L::x_pitch + unit * 64);
#pragma unroll
                                    for (int u = 0; u < 2; ++u) mma(d[u][c], a[2 * u][0], a[2 * u + 1][0], a[2 * u][1], a[2 * u + 1][1], b.x, b.y, d[u][c]);
#pragma unroll
                                    for (int u = 0; u < 2; ++u) mma(d[u][c], a[2 * u][2], a[2 * u + 1][2], a[2 * u][3], a[2 * u + 1][3], b.z, b.w, d[u][c]);
                                }
                            }
#pragma unroll
                            for (int u = 0; u < 2; ++u)
#pragma unroll
                                for (int c = 0; c < NT; ++c)
#pragma unroll
                                    for (int e = 0; e < 4; ++e) {
                                        const float by = sc[2 * u + (e >> 1)];
                                        run[u][c][e] = j ? fmaf(by, d[u][c][e], run[u][c][e]) : by * d[u][c][e];
                                    }
                        }
#pragma unroll
                        for (int c = 0; c < NT; ++c) {
                            const float by[2] = {f[8 * c * L::seg_runs + h], f[(8 * c + 1) * L::seg_runs + h]};  // of columns 2 t and 2 t + 1
#pragma unroll
                            for (int u = 0; u < 2; ++u)
#pragma unroll
                                for (int e = 0; e < 4; ++e) acc[u][c][e] = fmaf(by[e & 1], run[u][c][e], acc[u][c][e]);
                        }
                    }
                }
                if (++buffer == kStages) buffer = 0;
            }
        }
        if (ks > 1) {  // the first warp of each tile adds up the others' sums, in their order; they lie over the last columns
            __syncthreads();
            float4* red = reinterpret_cast<float4*>(smem + L::x_at + ((pass * segs + segs - 1) & 1) * L::cols * L::x_pitch) + warp * 2 * NT * 32 + lane;
            if (slot) {
#pragma unroll
                for (int u = 0; u < 2; ++u)
#pragma unroll
                    for (int c = 0; c < NT; ++c) red[(u * NT + c) * 32] = make_float4(acc[u][c][0], acc[u][c][1], acc[u][c][2], acc[u][c][3]);
            }
            __syncthreads();
            if (!slot) {
                for (int o = 1; o < ks; ++o)
#pragma unroll
                    for (int u = 0; u < 2; ++u)
#pragma unroll
                        for (int c = 0; c < NT; ++c) {
                            const float4 v = red[(o * 2 * NT + u * NT + c) * 32];
                            acc[u][c][0] += v.x, acc[u][c][1] += v.y, acc[u][c][2] += v.z, acc[u][c][3] += v.w;
                        }
            }
        }
        done(pass, acc);
    }
    cp_wait<0>();
}

// CTAs along the rows, for `blocks` blocks of columns: all SMs, as far as there are tiles of 32 rows, and warps that share
// a tile along K: the number that leaves a CTA the least to do (1,024 x 7,168 for one row: 12 us, 27 with a warp per tile).
struct Split {
    int ctas, ks;
};
template <typename L> Split split_rows(int tiles, int blocks, int K) {
    const int stages = (K + kStageK - 1) / kStageK, least_ctas = (tiles + L::W - 1) / L::W;
    Split s;
    s.ctas = 152 / blocks > least_ctas ? 152 / blocks : least_ctas < 152 ? least_ctas : 152;
    if (s.ctas > tiles) s.ctas = tiles;
    const int each = (tiles + s.ctas - 1) / s.ctas;
    s.ks = 1;
    int64_t least = INT64_MAX;
    for (int ks = 1; ks <= L::most_ks && L::W % ks == 0; ks *= 2) {
        const int64_t per = L::W / ks, t = ((each + per - 1) / per) * ((stages + ks - 1) / ks);
        if (t < least) least = t, s.ks = ks;
    }
    return s;
}

}  // namespace few
}  // namespace kda
