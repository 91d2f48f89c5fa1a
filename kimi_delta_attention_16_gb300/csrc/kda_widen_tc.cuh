// kda_widen_tc.cuh -- products of e2m1 weights with many rows of bf16 on tcgen05.mma kind::f16: weights become bf16 on
// their way from shared to tensor memory, which is exact (a code times a power of two), rows are read as they are.
//
// With many rows the digits of kda_few_tc.cuh cost more than they save: a row's eight columns are 4 bytes per element that
// every CTA moves into shared memory and reads from there again, 2 here.  Weights are the operand in tensor
// memory, so that shared memory holds and passes on their codes only, half a byte each.
//
// Warps of a CTA: 0 and 3 feed two rings by TMA, 128 elements of N columns and codes of 256 elements of 128 rows (a swizzled tile
// of 128-byte rows each); 1 issues the products; 4 to 19 widen codes, four warps 64 of every 256 elements, a thread a row (its
// lane of tensor memory), into a ring of four places of 128 elements, and carry the sums out at the end.
//
// Widening: three bits of a code, put at bits 6 to 8 of a bf16, are its value times 2^-126 (e2m1's subnormals are bf16's
// there), so one product with 2^(byte - 1) ends it; bytes above 128 need a second.
//
// Sums stay in one accumulator, which every instruction (16 elements) cuts off instead of rounding: 2^-23 of the sum of
// magnitudes at most, and all in one direction where products have one sign.  So a CTA takes kMostK elements at most: 2^-12 of
// the sum of magnitudes, an eighth of what rounding the result to bf16 costs - and so C is bf16 here, fp32 takes digits.
// Parts of longer rows are added up in fp32 by the cluster; rows longer than a cluster takes go to the digits.  Measured, 19,456 x K,
// 130 rows, products of one sign, all results together: 5e-6 too small at K = 7,168, 1.5e-5 at 16,384, and with one accumulator
// whatever the length 8.3e-5 at 65,536, 2.1e-4 at 131,072, 3.9e-3 at 2^20; random signs a twentieth of that.
// (kMostK = 16,384: 20,000 elements in 121 us instead of 111, 65,536 in 445 instead of 338.)
#pragma once

#include "kda_few_tc.cuh"

namespace kda {
namespace widetc {

using namespace tc;
using fewtc::arrive;
using fewtc::tma_2d;

constexpr int kThreads = 640;
constexpr int kSubK = 64, kRoundK = 128, kCodesK = 256, kPlaces = 4;
constexpr int kMostK = 32768;  // of one accumulator
constexpr int kMostRanks = 8;
static_assert(kMostK % fewtc::kStageK == 0, "slices are whole runs");
inline int least_ranks(int K) { return (K + kMostK - 1) / kMostK; }
constexpr uint32_t kCodes = few::kTileRows * (kCodesK / 2);

template <int N> struct Shape {
    static constexpr uint32_t sub = N * kSubK * 2, round = 2 * sub;  // bytes of 64 and 128 elements of the columns
    static constexpr int codes = N == 256 ? 2 : 4, rounds = N == 256 ? 3 : 5;
    static constexpr int places_at = N, tmem = 512;
    static constexpr uint32_t ring = codes * kCodes + rounds * round;
    static constexpr uint32_t red = N * few::kRedPitch * 4;      // the sums lie over the rings
    static_assert(codes <= 8 && rounds <= 8, "barriers");
    static_assert(red <= ring, "the sums fit over the rings");
    static_assert(places_at + kPlaces * kRoundK / 2 <= tmem, "accumulator and widened weights");
    static constexpr uint32_t smem = ring + 1024;
    // CTAs of a cluster wait for one another and for tensor memory.  They hold all of it here, so none that waits in the
    // same way (kda_few_tc.cuh: 90 KB at least) may fit beside them on an SM.
    static_assert(smem > 140 * 1024 && smem <= 227 * 1024, "shared memory of an SM");
};

struct Barriers {
    uint64_t codes_full[8], codes_empty[8], full[8], empty[8], place_full[kPlaces], place_empty[kPlaces], sums;
    uint32_t tmem;
    int failed;
};

template <int N> __device__ __forceinline__ void start(Barriers& bar) {
    using S = Shape<N>;
    if (threadIdx.x / 32 == 2) {
        tmem_alloc(&bar.tmem, S::tmem);
        tmem_relinquish();
    }
    if (threadIdx.x == 0) {
        for (int s = 0; s < 8; ++s) {
            mbar_init(&bar.codes_full[s], 1);
            mbar_init(&bar.codes_empty[s], 16);
            mbar_init(&bar.full[s], 1);
            mbar_init(&bar.empty[s], 1);
        }
        for (int s = 0; s < kPlaces; ++s) {
            mbar_init(&bar.place_full[s], 8);
            mbar_init(&bar.place_empty[s], 1);
        }
        mbar_init(&bar.sums, 1);
        bar.failed = 0;
        fence_mbar_init();
    }
    fence_before_sync();
    __syncthreads();
    fence_after_sync();
}
// Every thread has passed a barrier since its last use of tensor memory.
template <int N> __device__ __forceinline__ void finish(Barriers& bar, int* d_status) {
    if (threadIdx.x == 0 && bar.failed) flag_status(d_status, KDA_ERR_TIMEOUT);
    if (threadIdx.x / 32 == 2) tmem_dealloc(bar.tmem, Shape<N>::tmem);
}

__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

// 32 codes of a row under one scale byte as 16 pairs of bf16: of eight codes (0,4), (1,5), (2,6), (3,7), the order in which
// k_widen_rows lays out the columns.  Shifts to the left are products, which have a pipe of their own.
__device__ __forceinline__ void widen(const uint4& codes, uint32_t byte, bool large, uint32_t (&out)[16]) {
    const uint32_t w[4] = {codes.x, codes.y, codes.z, codes.w};
    constexpr uint32_t kSign = 0x80008000u, kValue = 0x01c001c0u;
    // 2^(byte - 1) where bf16 has it (bytes to 128), else 2^127 and then 2^(byte - 128)
    const uint32_t by = min(byte + 126u, 254u) * 0x00800080u;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t h = w[i] >> 6;
        out[4 * i] = mul_bf16x2((w[i] * 4096u & kSign) | (w[i] * 64u & kValue), by);
        out[4 * i + 1] = mul_bf16x2((w[i] * 256u & kSign) | (w[i] * 4u & kValue), by);
        out[4 * i + 2] = mul_bf16x2((w[i] * 16u & kSign) | (h * 16u & kValue), by);
        out[4 * i + 3] = mul_bf16x2((w[i] & kSign) | (h & kValue), by);
    }
    if (large) {
        const uint32_t more = (byte > 128u ? byte - 1u : 127u) * 0x00800080u;
#pragma unroll
        for (int i = 0; i < 16; ++i) out[i] = mul_bf16x2(out[i], more);
    }
}

struct Tile {
    const CUtensorMap *w, *x;  // codes in boxes of 128 rows, rows of x in boxes of N
    int row0, c0;
    const uint8_t* scales;     // [.][K / 32]
    int last_row;              // scales of rows past it are read as its own
    int K, k0, k1;             // K a multiple of 32; k0 and, except at K's end, k1 of 256
};

// red[column][128 rows] = the tile's sums over [k0, k1).  `ring` is 1024-byte aligned; red lies over it.  Ends with a barrier of
// the CTA.  After a wait that ran out bar.failed is set and red holds nothing of use.
template <int N> __device__ __forceinline__ void product(uint8_t* ring, Barriers& bar, const Tile& t, float* red) {
    using S = Shape<N>;
    const int warp = fewtc::warp_index(), lane = threadIdx.x & 31;
    const int subs = (t.k1 - t.k0 + kSubK - 1) / kSubK, rounds = (subs + 1) / 2, blocks = (subs + 3) / 4;
    const uint32_t base = smem_u32(ring), cols = base + S::codes * kCodes, tm = bar.tmem;
    if ((warp == 0 || warp == 3) && lane == 0) {
        // columns and codes, each as far ahead as its own ring goes; codes need not wait for the kernel that writes the columns
        const bool codes = warp == 3;
        if (!codes) few::wait_for_kernel_before();
        uint64_t *full = codes ? bar.codes_full : bar.full, *empty = codes ? bar.codes_empty : bar.empty;
        const int stages = codes ? S::codes : S::rounds, last = codes ? blocks : rounds;
        for (int i = 0; i < last; ++i) {
            const int s = i % stages;
            if (!mbar_wait(&empty[s], ((i / stages) & 1u) ^ 1u)) {
                bar.failed = 1;
                // copies still in flight: wait for them before the shared memory is used for anything else
                for (int j = max(i - stages, 0); j < i; ++j) mbar_wait(&full[j % stages], (j / stages) & 1u);
                break;
            }
            if (codes) {
                mbar_expect_tx(&full[s], kCodes);
                tma_2d(base + s * kCodes, t.w, (t.k0 + i * kCodesK) / 2, t.row0, &full[s]);
            } else {
                const bool both = 2 * i + 1 < subs;
                mbar_expect_tx(&full[s], both ? S::round : S::sub);
                tma_2d(cols + s * S::round, t.x, t.k0 + i * kRoundK, t.c0, &full[s]);
                if (both) tma_2d(cols + s * S::round + S::sub, t.x, t.k0 + i * kRoundK + kSubK, t.c0, &full[s]);
            }
        }
    } else if (warp == 1) {
        const uint64_t first = desc_sw128(cols, 16, 1024);
        few::wait_for_kernel_before();  // its time does not count against a wait's deadline
        int s = 0;
        uint32_t phase = 0;
        for (int i = 0; i < rounds; ++i) {
            const int place = i % kPlaces;
            if (!fewtc::warp_wait(&bar.full[s], phase) || !fewtc::warp_wait(&bar.place_full[place], (i / kPlaces) & 1u)) {
                bar.failed = 1;
                break;
            }
            fence_after_sync();
            if (fewtc::elected()) {
                const uint64_t b = first + s * (S::round >> 4);
                const uint32_t a = tm + S::places_at + place * (kRoundK / 2);
#pragma unroll
                for (int kk = 0; kk < 8; ++kk)
                    if (kk < 4 || 2 * i + 1 < subs)
                        mma_ts(tm, a + 8 * kk, b + (kk >> 2) * (S::sub >> 4) + 2 * (kk & 3), idesc_bf16(128, N, false, false), (i | kk) != 0);
                mma_commit(&bar.empty[s]);
                mma_commit(&bar.place_empty[place]);
                if (i == rounds - 1) mma_commit(&bar.sums);
            }
            __syncwarp();
            if (++s == S::rounds) s = 0, phase ^= 1u;
        }
    } else if (warp >= 4) {
        const int q = warp & 3, set = (warp - 4) >> 2, r = 32 * q + lane;
        const uint32_t quadrant = (uint32_t)q * 32 << 16;
        const int64_t pitch = t.K >> 5;
        const uint8_t* scales = t.scales + min(t.row0 + r, t.last_row) * pitch;
        const auto load_scales = [&](int g) -> uint32_t {  // the two bytes of this set's 64 elements, 2^0 past the last
            const int k = t.k0 + g * kCodesK + set * kSubK;
            if (k >= t.k1) return 0x7f7fu;
            return scales[k >> 5] | (k + 32 < t.k1 ? (uint32_t)scales[(k >> 5) + 1] : 0x7fu) << 8;
        };
        uint32_t ahead[2] = {load_scales(0), load_scales(1)};
        bool ok = true;
        for (int g = 0; g < blocks && ok; ++g) {
            const uint32_t two = ahead[0];
            ahead[0] = ahead[1];
            ahead[1] = load_scales(g + 2);
            const int s = g % S::codes, i = 4 * g + set, round = i >> 1, place = round % kPlaces;
            if (lane == 0) ok = mbar_wait(&bar.codes_full[s], (g / S::codes) & 1u);
            ok = __shfl_sync(0xffffffffu, ok ? 1 : 0, 0);
            if (!ok) break;
            const uint8_t* row = ring + s * kCodes + r * 128;
            const uint4 a = *reinterpret_cast<const uint4*>(row + (((2 * set) ^ (r & 7)) << 4));
            const uint4 b = *reinterpret_cast<const uint4*>(row + (((2 * set + 1) ^ (r & 7)) << 4));
            const uint32_t ea = two & 255u, eb = two >> 8;
            const bool large = __any_sync(0xffffffffu, max(ea, eb) > 128u);
            uint32_t va[16], vb[16];
            widen(a, ea, large, va);
            widen(b, eb, large, vb);
            __syncwarp();
            if (lane == 0) arrive(&bar.codes_empty[s]);
            if (round >= rounds) continue;
            if (2 * g == kPlaces) few::wait_for_kernel_before();  // from here on places come back as products end
            if (lane == 0) ok = mbar_wait(&bar.place_empty[place], ((round / kPlaces) & 1u) ^ 1u);
            ok = __shfl_sync(0xffffffffu, ok ? 1 : 0, 0);
            if (!ok) break;
            if (i < subs) {
                fence_after_sync();
                const uint32_t at = tm + quadrant + S::places_at + place * (kRoundK / 2) + (set & 1) * (kSubK / 2);
                tmem_st16(at, va);
                tmem_st16(at + 16, vb);
                tmem_st_wait();
                fence_before_sync();
            }
            __syncwarp();
            if (lane == 0) arrive(&bar.place_full[place]);
        }
        few::wait_for_kernel_before();
        if (lane == 0 && ok) ok = mbar_wait(&bar.sums, 0u);
        ok = __shfl_sync(0xffffffffu, ok ? 1 : 0, 0);
        if (ok) {
            fence_after_sync();
#pragma unroll 2
            for (int n = set * 16; n < N; n += 64) {
                uint32_t v[16];
                tmem_ld16(tm + quadrant + n, v);
                tmem_ld_wait();
#pragma unroll
                for (int i = 0; i < 16; ++i) red[(n + i) * few::kRedPitch + r] = __uint_as_float(v[i]);
            }
        } else if (lane == 0) {
            bar.failed = 1;
        }
        fence_before_sync();
    }
    __syncthreads();
    fence_after_sync();
}

}  // namespace widetc
}  // namespace kda
