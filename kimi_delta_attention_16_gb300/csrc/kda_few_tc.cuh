// kda_few_tc.cuh -- products of e2m1 weights with a few columns on the tensor cores' block-scaled instruction for
// 4-bit operands (tcgen05.mma kind::mxf4): codes and their scale bytes go to the tensor cores as they are stored, so
// nothing is widened or multiplied by a scale in registers, and the time is that of reading the codes.
//
//   rows (M = 128)  e2m1 codes of the weights, 256 elements (128 bytes) of a row per stage
//   columns (N)     the tokens' values as digits: with 2^e the power of two that brings the largest of 32 values to at most
//                   4, v 2^-e = d_0 + d_1 / 8 + d_2 / 64 + ... with whole digits from -4 to 4, each of which is an e2m1
//                   value.  Eight digits leave at most 2^-22 2^e, 2^-23 of the 32 values' largest: as good as an fp32 sum
//                   keeps them.  Digit t is a column of its own under the scale e - 3 t; a token's eight columns
//                   are added up at the end.
//   scales          bytes (exponent + 127) in tensor memory: of rows 32 j + l, lane l, column j; an instruction takes 64
//                   elements and two of a word's four bytes, which its descriptor names; the same in all four quadrants
//
// Warps of a CTA: 0 feeds a ring of stages by TMA, 1 issues the products, 4 to 7 bring the scales of 512 elements at a time
// (each warp those of 32 rows, three such groups on their way, exchanged through shared memory) into a ring of three
// places in tensor memory, each its own quadrant, and carry the sums out at the end.  Weights and their scales are on
// their way before the kernel that writes the columns is done.  Every wait has a deadline (kda_tc_ptx.cuh).
//
// The wider instruction kind::mxf8f6f4 would take e4m3 columns, two for a bf16 value, but reads 4-bit rows one byte per
// code: TMA spreads codes at 8 bytes a cycle and SM (2.3 TB/s in all, measured), registers cost more than the products.
#pragma once

#include "kda_few.cuh"
#include "kda_tc.cuh"
#include "kda_tc_ptx.cuh"

namespace kda {
namespace fewtc {

using namespace tc;

constexpr int kThreads = 256;
constexpr int kDigits = 8;                             // columns of a token
constexpr int kStageK = 256, kGroupK = 512, kSlots = 3;
constexpr uint32_t kRowBytes = kStageK / 2;            // of a row, weight or column, in a stage
constexpr uint32_t kTileA = few::kTileRows * kRowBytes;

template <int N> struct Shape {
    static constexpr int tokens = N / kDigits;
    static constexpr uint32_t stage = kTileA + N * kRowBytes;
    static constexpr int stages = N <= 32 ? 5 : N == 64 ? 4 : N == 128 ? 3 : 4;
    static constexpr int per_sm = N <= 128 ? 2 : 1;
    // Columns of tensor memory with the scales of N columns over 128 elements, and the distance between two such sets:
    // the instruction takes a set only at a multiple of four columns.
    static constexpr int nb = N < 32 ? 1 : N / 32, set = nb < 4 ? 4 : nb;
    static constexpr int group = 16 + 4 * set;                  // of one place of the scales' ring
    static_assert(group % 4 == 0 && set % 4 == 0, "sets of scales start at multiples of four columns");
    static constexpr int scales_at = N < 32 ? 32 : N;
    static constexpr int need = scales_at + kSlots * group;
    static constexpr int tmem = need <= 128 ? 128 : need <= 256 ? 256 : 512;
    static constexpr uint32_t red = tokens * few::kRedPitch * 4;  // the sums lie over the ring
    static constexpr uint32_t ring = stages * stage;
    static_assert(red <= ring, "the sums fit over the ring");
    static constexpr int words = 128 + 4 * nb;                  // rows and tokens whose scales are exchanged
    static constexpr uint32_t scales = 2 * words * 16;          // two groups
    static constexpr uint32_t smem = ring + scales + 1024;
};

struct Barriers {
    uint64_t full[5], empty[5], scales_full[kSlots], scales_empty[kSlots], sums;
    uint32_t tmem;
    int failed;
};

// e2m1 x e2m1 -> fp32 over 64 elements, one scale byte per 32 of each side; `byte`: the first of the two in a word.
__host__ __device__ constexpr uint32_t idesc_mxf4(int N, int byte) {
    return (1u << 7)                        // A: e2m1
           | (1u << 10)                     // B: e2m1
           | ((uint32_t)(N >> 3) << 17)
           | (1u << 23)                     // scales: powers of two
           | (8u << 24)                     // M = 128
           | ((uint32_t)byte << 4)          // of B's scale words
           | ((uint32_t)byte << 29);        // of A's
}
__device__ __forceinline__ void mma_mxf4(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t sa, uint32_t sb, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %6, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(sa), "r"(sb), "r"(accumulate)
        : "memory");
}
__device__ __forceinline__ void tma_2d(uint32_t dst, const CUtensorMap* map, int x, int y, uint64_t* bar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::
            "r"(dst), "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(smem_u32(bar))
        : "memory");
}
__device__ __forceinline__ void arrive(uint64_t* bar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_u32(bar)) : "memory");
}

// The warp that issues products runs as a whole, one lane of it issues: what an instruction takes is then known to be the same in all
// lanes and stays where the instruction takes it from.  Under a branch for one lane each product takes some 90 cycles
// to issue, more than most take to run.
__device__ __forceinline__ int warp_index() { return __shfl_sync(0xffffffffu, (int)threadIdx.x >> 5, 0); }
__device__ __forceinline__ bool elected() {
    uint32_t one;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(one));
    return one != 0;
}
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity) { return __all_sync(0xffffffffu, mbar_wait(bar, parity)); }

// What one product reads.  The tile's rows are two runs of 64.
struct Tile {
    const CUtensorMap *w, *b; // codes of the weights in boxes of 64 rows, digits of the columns in boxes of N
    int row0, row64;          // of the weights
    int token0;
    const uint8_t* w_scales;  // [.][K / 32]
    const uint8_t* b_scales;  // [.][K / 32], of the digits in front
    int last_row, last_token; // scales of rows and tokens past these are read as theirs
    int K, k0, k1;            // K a multiple of 32; k0 and, except at K's end, k1 of 256
};

// Scale words of four runs of 128 elements, from element k of a row (0 past the last element).
__device__ __forceinline__ uint4 load_scales(const uint8_t* row, int k, int k1, int aligned) {
    if (aligned >= 16 && (k & (kGroupK - 1)) == 0 && k + kGroupK <= k1) return *reinterpret_cast<const uint4*>(row + (k >> 5));
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int at = k + i * 128;
        w[i] = 0;
        if (aligned >= 4) {
            if (at < k1) w[i] = *reinterpret_cast<const uint32_t*>(row + (at >> 5));
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (at + 32 * j < k1) w[i] |= (uint32_t)row[(at >> 5) + j] << (8 * j);
        }
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ int alignment(const uint8_t* p, int64_t pitch) {
    const uint64_t v = reinterpret_cast<uint64_t>(p) | (uint64_t)pitch;
    return v % 16 == 0 ? 16 : v % 4 == 0 ? 4 : 1;
}
__device__ __forceinline__ void scale_warps_sync() { asm volatile("bar.sync 1, 128;" ::: "memory"); }

// A launch may begin beside the kernel in front of it (launch_kernel); it waits for what that one writes, the columns.
__device__ __forceinline__ void wait_for_columns() { few::wait_for_kernel_before(); }

// Once per CTA, before the first product.
template <int N> __device__ __forceinline__ void start(Barriers& bar) {
    using S = Shape<N>;
    if (threadIdx.x / 32 == 2) {
        tmem_alloc(&bar.tmem, S::tmem);
        tmem_relinquish();
    }
    if (threadIdx.x == 0) {
        for (int s = 0; s < S::stages; ++s) {
            mbar_init(&bar.full[s], 1);
            mbar_init(&bar.empty[s], 1);
        }
        for (int s = 0; s < kSlots; ++s) {
            mbar_init(&bar.scales_full[s], 4);
            mbar_init(&bar.scales_empty[s], 1);
        }
        mbar_init(&bar.sums, 1);
        bar.failed = 0;
        fence_mbar_init();
    }
    fence_before_sync();
    __syncthreads();
    fence_after_sync();
}

// Once per CTA, after the last: every thread has passed a barrier since its last use of tensor memory.
template <int N> __device__ __forceinline__ void finish(Barriers& bar, int* d_status) {
    if (threadIdx.x == 0 && bar.failed) flag_status(d_status, KDA_ERR_TIMEOUT);
    if (threadIdx.x / 32 == 2) tmem_dealloc(bar.tmem, Shape<N>::tmem);
}

struct Counters {  // of stages, places of scales and products so far: the barriers' phases follow from them
    uint32_t stage = 0, slot = 0, product = 0;
};

// red[token][128 rows] = the tile's sums over [k0, k1).  `ring` is 1024-byte aligned; red lies over it.  Ends with a
// barrier of the CTA.  After a wait that ran out bar.failed is set and red holds nothing of use.
template <int N> __device__ __forceinline__ void product(uint8_t* ring, Barriers& bar, const Tile& t, Counters& c, float* red) {
    using S = Shape<N>;
    const int warp = warp_index(), lane = threadIdx.x & 31;
    const int blocks = (t.k1 - t.k0 + kStageK - 1) / kStageK, groups = (blocks + 1) / 2;
    const uint32_t base = smem_u32(ring), tm = bar.tmem;
    if (warp == 0 && lane == 0) {
        const auto rows = [&](int kb, uint32_t s) {
            const int x = (t.k0 + kb * kStageK) / 2;
            mbar_expect_tx(&bar.full[s], S::stage);
            tma_2d(base + s * S::stage, t.w, x, t.row0, &bar.full[s]);
            tma_2d(base + s * S::stage + kTileA / 2, t.w, x, t.row64, &bar.full[s]);
        };
        const auto columns = [&](int kb, uint32_t s) {
            tma_2d(base + s * S::stage + kTileA, t.b, (t.k0 + kb * kStageK) / 2, t.token0 * kDigits, &bar.full[s]);
        };
        int issued = 0;
        bool failed = false;
        // the first round's weights, then - once they are written - its columns
        const int first = min(blocks, S::stages);
        for (int kb = 0; kb < first && !failed; ++kb) {
            const uint32_t i = c.stage + kb, s = i % S::stages;
            failed = !mbar_wait(&bar.empty[s], ((i / S::stages) & 1u) ^ 1u);
            if (!failed) {
                rows(kb, s);
                issued = kb + 1;
            }
        }
        wait_for_columns();
        for (int kb = 0; kb < issued; ++kb) columns(kb, (c.stage + kb) % S::stages);
        for (int kb = first; kb < blocks && !failed; ++kb) {
            const uint32_t i = c.stage + kb, s = i % S::stages;
            failed = !mbar_wait(&bar.empty[s], ((i / S::stages) & 1u) ^ 1u);
            if (!failed) {
                rows(kb, s);
                columns(kb, s);
                issued = kb + 1;
            }
        }
        if (failed) {
            bar.failed = 1;
            // copies still in flight: wait for them before the shared memory is used for anything else
            for (int kb = issued > S::stages ? issued - S::stages : 0; kb < issued; ++kb)
                mbar_wait(&bar.full[(c.stage + kb) % S::stages], ((c.stage + kb) / S::stages) & 1u);
        }
    } else if (warp == 1) {
        const uint64_t rows = desc_sw128(base, 16, 1024), columns = desc_sw128(base + kTileA, 16, 1024);
        wait_for_columns();  // the time of the kernel in front does not count against a wait's deadline
        for (int kb = 0; kb < blocks; ++kb) {
            const uint32_t i = c.stage + kb, s = i % S::stages, gi = c.slot + kb / 2, slot = gi % kSlots;
            if (!warp_wait(&bar.full[s], (i / S::stages) & 1u) ||
                ((kb & 1) == 0 && !warp_wait(&bar.scales_full[slot], (gi / kSlots) & 1u))) {
                bar.failed = 1;
                break;
            }
            fence_after_sync();
            if (elected()) {
                const uint32_t at = s * (S::stage >> 4), sf = tm + S::scales_at + slot * S::group;
#pragma unroll
                for (int kk = 0; kk < 4; ++kk) {
                    const int set = 2 * (kb & 1) + (kk >> 1);  // of 128 elements
                    mma_mxf4(tm, rows + at + 2 * kk, columns + at + 2 * kk, idesc_mxf4(N, 2 * (kk & 1)), sf + 4 * set, sf + 16 + S::set * set,
                             (kb | kk) != 0);
                }
                mma_commit(&bar.empty[s]);
                if ((kb & 1) || kb == blocks - 1) mma_commit(&bar.scales_empty[slot]);
            }
            __syncwarp();
        }
        if (elected()) mma_commit(&bar.sums);
        __syncwarp();
    } else if (warp >= 4) {
        // This warp's 32 rows, and the tokens whose scales it brings: eight lanes stand for one token.
        const int q = warp & 3;
        const uint32_t quadrant = (uint32_t)q * 32 << 16;
        const int64_t pitch = t.K >> 5;
        const int wa = alignment(t.w_scales, pitch), wb = alignment(t.b_scales, pitch);
        constexpr int kAhead = 3;
        const uint8_t* ra = t.w_scales + min((q < 2 ? t.row0 : t.row64 - 64) + 32 * q + lane, t.last_row) * pitch;
        const int token = 32 * q + lane;  // of at most 32
        const uint8_t* rb = t.b_scales + min(t.token0 + token, t.last_token) * pitch;
        uint4* place = reinterpret_cast<uint4*>(ring + S::ring);  // [2][rows, then tokens]
        uint4 av[kAhead], bv[kAhead];
        auto load_a = [&](int g, int i) {
            if (g < groups) av[i] = load_scales(ra, t.k0 + g * kGroupK, t.k1, wa);
        };
        auto load_b = [&](int g, int i) {
            if (g < groups && token < 4 * S::nb) bv[i] = load_scales(rb, t.k0 + g * kGroupK, t.k1, wb);
        };
#pragma unroll
        for (int i = 0; i < kAhead; ++i) load_a(i, i);
        wait_for_columns();
#pragma unroll
        for (int i = 0; i < kAhead; ++i) load_b(i, i);
        bool failed = false;
        const uint32_t down = 0x03030303u * (lane & 7);  // a digit's scale is 2^-3 of the one in front
        for (int g0 = 0; g0 < groups; g0 += kAhead) {
#pragma unroll
            for (int i = 0; i < kAhead; ++i) {
                const int g = g0 + i;
                if (g >= groups) break;
                uint4* here = place + (g & 1) * S::words;
                here[32 * q + lane] = av[i];
                if (token < 4 * S::nb) here[128 + token] = bv[i];
                load_a(g + kAhead, i);
                load_b(g + kAhead, i);
                scale_warps_sync();  // and nobody is two groups behind: each has read the place that comes next
                const uint32_t gi = c.slot + g, slot = gi % kSlots, at = tm + quadrant + S::scales_at + slot * S::group;
                if (!failed) {
                    bool ok = true;
                    if (lane == 0) ok = mbar_wait(&bar.scales_empty[slot], ((gi / kSlots) & 1u) ^ 1u);
                    failed = !__shfl_sync(0xffffffffu, ok ? 1 : 0, 0);
                }
                if (failed) continue;
                fence_after_sync();
                {
                    const uint4 r0 = here[lane], r1 = here[32 + lane], r2 = here[64 + lane], r3 = here[96 + lane];
                    const uint32_t a[16] = {r0.x, r1.x, r2.x, r3.x, r0.y, r1.y, r2.y, r3.y, r0.z, r1.z, r2.z, r3.z, r0.w, r1.w, r2.w, r3.w};
                    tmem_st16(at, a);
                }
#pragma unroll
                for (int h = 0; h < S::nb; h += 4) {  // four columns of the sets at a time: four tokens each
                    uint4 b[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        b[j] = h + j < S::nb ? here[128 + 4 * (h + j) + (lane >> 3)] : make_uint4(0, 0, 0, 0);
                        b[j].x -= down, b[j].y -= down, b[j].z -= down, b[j].w -= down;
                    }
                    tmem_st4(at + 16 + h, make_uint4(b[0].x, b[1].x, b[2].x, b[3].x));
                    tmem_st4(at + 16 + S::set + h, make_uint4(b[0].y, b[1].y, b[2].y, b[3].y));
                    tmem_st4(at + 16 + 2 * S::set + h, make_uint4(b[0].z, b[1].z, b[2].z, b[3].z));
                    tmem_st4(at + 16 + 3 * S::set + h, make_uint4(b[0].w, b[1].w, b[2].w, b[3].w));
                }
                tmem_st_wait();
                fence_before_sync();
                __syncwarp();
                if (lane == 0) arrive(&bar.scales_full[slot]);
            }
        }
        bool ok = !failed;
        if (lane == 0 && ok) ok = mbar_wait(&bar.sums, c.product & 1u);
        ok = __shfl_sync(0xffffffffu, ok ? 1 : 0, 0);
        if (ok) {
            fence_after_sync();
#pragma unroll 2
            for (int n = 0; n < N; n += 16) {
                uint32_t v[16];
                tmem_ld16(tm + quadrant + n, v);
                tmem_ld_wait();
#pragma unroll
                for (int i = 0; i < 16; i += kDigits) {
                    float sum = __uint_as_float(v[i + kDigits - 1]);  // the smallest part first
#pragma unroll
                    for (int j = kDigits - 2; j >= 0; --j) sum += __uint_as_float(v[i + j]);
                    red[(n + i) / kDigits * few::kRedPitch + 32 * q + lane] = sum;
                }
            }
        } else if (lane == 0) {
            bar.failed = 1;
        }
        fence_before_sync();
    }
    c.stage += blocks;
    c.slot += groups;
    ++c.product;
    __syncthreads();
    fence_after_sync();
}

// ------------------------------------------------------------------ columns from values
// The largest magnitude of 32 values, as fp32 bits (four lanes share them, eight each; the whole warp calls it).
__device__ __forceinline__ uint32_t largest_of_32(const float (&r)[8]) {
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) top = max(top, __float_as_uint(r[i]) & 0x7fffffffu);
    top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
    return max(top, __shfl_xor_sync(0xffffffffu, top, 2));
}

// The scale of the digits in front goes down to 2^-105, so that the eighth digit's is one too: values below 2^-103 lose
// digits, what is left of them is off by 2^-127 at most.  Rows of x that are as small throughout go to direct(); hidden values
// of an expert have no such way (their rows come together from many CTAs) and are off by that much.
constexpr int kLowestByte = 22;
constexpr uint32_t kLowestTop = (uint32_t)(kLowestByte + 2) << 23;

// The digits of eight values from element k of a token's row, with the largest of their 32 (lanes without `in` write
// nothing): rows token * 8 .. of the digits' tensor [.][K / 2], and the scale of the digits in front, NaN for values that
// are not finite.
__device__ __forceinline__ void put_digits(float (&r)[8], uint32_t top, bool in, int64_t token, int k, int K, uint8_t* digits, uint8_t* scales) {
    const bool finite = top < 0x7f800000u;
    // the smallest power of two that keeps the largest magnitude within 4
    const int byte = max((int)((top + 0x7fffffu) >> 23) - 2, kLowestByte);
    const float by = __uint_as_float((uint32_t)(254 - byte) << 23);  // byte is at most 253
#pragma unroll
    for (int i = 0; i < 8; ++i) r[i] = finite ? r[i] * by : 0.f;
    uint32_t* to = reinterpret_cast<uint32_t*>(digits + (token * kDigits * K + k) / 2);
#pragma unroll
    for (int t = 0; t < kDigits; ++t) {
        float d[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            d[i] = rintf(r[i]);
            r[i] = (r[i] - d[i]) * 8.f;  // exact
        }
        uint32_t w;
        asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
            "cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n\tcvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n\t"
            "cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n\tcvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n\t"
            "mov.b32 %0, {b0, b1, b2, b3};\n\t}"
            : "=r"(w) : "f"(d[0]), "f"(d[1]), "f"(d[2]), "f"(d[3]), "f"(d[4]), "f"(d[5]), "f"(d[6]), "f"(d[7]));
        if (in) to[(int64_t)t * (K / 8)] = w;
    }
    if (in && (k & 31) == 0) scales[(token * K + k) >> 5] = finite ? (uint8_t)byte : (uint8_t)255;
}

// The same with one value per lane, 32 in a row from element k - lane; `top` is their largest.
__device__ __forceinline__ void put_digits_of_lanes(float v, uint32_t top, bool in, int64_t token, int k, int K, uint8_t* digits, uint8_t* scales) {
    const bool finite = top < 0x7f800000u;
    const int byte = max((int)((top + 0x7fffffu) >> 23) - 2, kLowestByte), lane = threadIdx.x & 31;
    float r = finite ? v * __uint_as_float((uint32_t)(254 - byte) << 23) : 0.f;
#pragma unroll
    for (int t = 0; t < kDigits; ++t) {
        const float d = rintf(r);
        r = (r - d) * 8.f;
        // 0, 1, 2, 3, 4 are the codes 0, 2, 4, 5, 6; bit 3 is the sign
        const uint32_t code = (0x65420u >> (4 * (int)fabsf(d)) & 15u) | (d < 0.f ? 8u : 0u);
        // eight lanes' codes in one word
        uint32_t w = code << (4 * (lane & 7));
        w |= __shfl_xor_sync(0xffffffffu, w, 1);
        w |= __shfl_xor_sync(0xffffffffu, w, 2);
        w |= __shfl_xor_sync(0xffffffffu, w, 4);
        if (in && (lane & 7) == 0) *reinterpret_cast<uint32_t*>(digits + ((token * kDigits + t) * K + k) / 2) = w;
    }
    if (in && lane == 0) scales[(token * K + k) >> 5] = finite ? (uint8_t)byte : (uint8_t)255;
}

// Digits of bf16 rows: token p is row of[p] / per of x (p itself without `of`).
cudaError_t launch_digits(const bf16* x, int64_t xs, bool wide, const int* of, int per, int tokens, int K, uint8_t* digits, uint8_t* scales,
                          cudaStream_t s);

// The rows themselves, for bf16 weights.
cudaError_t launch_rows(const bf16* x, int64_t xs, bool wide, const int* of, int per, int tokens, int K, bf16* rows, cudaStream_t s);

// Bytes of the digits of so many values, and of their scales.
inline size_t digits_bytes(int64_t tokens, int64_t K) { return (size_t)tokens * kDigits * K / 2; }
inline size_t digit_scales_bytes(int64_t tokens, int64_t K) { return (size_t)tokens * (K / 32); }

struct Maps {
    CUtensorMap w, b;
};
inline bool encode_maps(Maps* m, const void* codes, int64_t rows, const uint8_t* digits, int64_t tokens, int K, int box) {
    return encode_tensor_map_2d_as(&m->w, CU_TENSOR_MAP_DATA_TYPE_UINT8, codes, K / 2, rows, K / 2, kRowBytes, 64, true) &&
           encode_tensor_map_2d_as(&m->b, CU_TENSOR_MAP_DATA_TYPE_UINT8, digits, K / 2, tokens * kDigits, K / 2, kRowBytes, box, true);
}

// The same for bf16 weights and columns, in boxes of 64 elements.
inline bool encode_maps_bf16(Maps* m, const void* w, int64_t rows, const void* columns, int64_t n, int K, int box) {
    return encode_tensor_map_2d_as(&m->w, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, w, K, rows, 2 * (uint64_t)K, 64, 64, true) &&
           encode_tensor_map_2d_as(&m->b, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, columns, K, n, 2 * (uint64_t)K, 64, box, true);
}

// One product by itself, for a sum that came out as NaN or infinite: a row of x that digits do not hold (values that are not
// finite, or all tiny), or sums next to the end of fp32, where the digits in front, rounded up, pass it.  An eighth of the
// weight times x, so that only a product that overflows does.
static __device__ __noinline__ float direct(const uint8_t* codes, const uint8_t* scales, const bf16* x, int K) {
    float sum = 0.f;
    for (int g = 0; g < K / 32; ++g) {
        const float s = __uint_as_float((uint32_t)scales[g] << 23);
        for (int i = 0; i < 32; ++i) {
            const uint32_t c = codes[(g * 32 + i) >> 1] >> (4 * (i & 1)) & 15u;
            const float eighth = (c & 6u) ? __uint_as_float(((123u + ((c >> 1) & 3u)) << 23) | ((c & 1u) << 22)) : 0.0625f * (c & 1u);
            sum = fmaf(((c & 8u) ? -eighth : eighth) * s, to_f(x[g * 32 + i]), sum);
        }
    }
    return 8.f * sum;
}

// The part of K that a rank of a cluster takes, in whole runs of 256.
__device__ __forceinline__ void slice_of(int K, int rank, int ranks, int& k0, int& k1) {
    const int runs = (K + kStageK - 1) / kStageK;
    k0 = (int)((int64_t)runs * rank / ranks) * kStageK;
    k1 = min(K, (int)((int64_t)runs * (rank + 1) / ranks) * kStageK);
}

// The rows of a tile that a rank joins and writes, in fours.
__device__ __forceinline__ void rows_of(int rank, int ranks, int& r0, int& r1) {
    r0 = 32 * rank / ranks * 4;
    r1 = 32 * (rank + 1) / ranks * 4;
}

// Four rows of a token's joined sums, the ranks' parts on their way together and added in their order.
__device__ __forceinline__ float4 joined4(const float* red, int ranks, int token, int r) {
    const float* mine = red + token * few::kRedPitch + r;
    if (ranks == 1) return *reinterpret_cast<const float4*>(mine);
    float4 v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if (i < ranks) v[i] = *reinterpret_cast<const float4*>(cooperative_groups::this_cluster().map_shared_rank(mine, i));
#pragma unroll
    for (int i = 1; i < 8; ++i)
        if (i < ranks) v[0].x += v[i].x, v[0].y += v[i].y, v[0].z += v[i].z, v[0].w += v[i].w;
    return v[0];
}

// CTAs of a cluster that share a tile's K: the number that leaves the busiest SM the least to do, in runs of 256 elements,
// where the CTAs that run side by side take about `overhead` runs' time to start and to join; `at_least` of them.  In a captured
// graph, one row: 12,288 x 7,168 in 14.0 us by one CTA per tile, 12.7 by three (the rule), 21.0 by eight; 1,024 x 7,168 in 12.7, 8.5
// and 6.9 (the rule).  Whole ranks per tile only: 32 rows of 12,288 x 7,168 keep one CTA per tile, 96 on 152 SMs (18.6 us; two 24.6).
inline int cluster_ranks(int64_t tiles, int K, int per_sm, int overhead, int at_least = 1) {
    const int runs = (K + 255) / 256;
    int best = at_least;
    int64_t least = INT64_MAX;
    for (int r = at_least; r <= 8 && r <= runs; ++r) {
        const int64_t on_one = (tiles * r + 151) / 152;
        const int64_t t = on_one * ((runs + r - 1) / r) + (on_one + per_sm - 1) / per_sm * overhead;
        if (t < least) least = t, best = r;
    }
    return best;
}

}  // namespace fewtc
}  // namespace kda
