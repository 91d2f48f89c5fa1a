// kda_moe_tc.cuh -- the experts' products on the tensor cores, for weights in e2m1 (kda_few_tc.cuh) and in bf16: CTAs that
// stay and walk over tiles of 128 rows of the experts in use.
//
// As in kda_few_tc.cuh warp 0 feeds a ring of stages by TMA, warp 1 issues the products, warps 4 to 7 bring scales (e2m1
// only).  Warps 8 to 11 carry sums out of one accumulator in tensor memory while the next tile fills another, so
// copies never pause between tiles.  A stage is 128 bytes of every row: 256 elements of e2m1, 64 of bf16.
//
// bf16 weights take bf16 columns on tcgen05.mma kind::f16; an fp32 hidden value is the sum of three bf16 terms, columns of
// their own (and one of zeros), added up at the end.  That instruction cuts its sums off where the accumulator ends: over
// 2,048 elements (128 instructions) the result is off by 5.7e-6.  So a bf16 tile is carried out every two stages (8
// instructions) and added up in fp32: 4.0e-7, and 83.7 us for four tokens of 6 of 64 experts (2,048 x 1,408) against 82.1
// for whole tiles (every four stages: 7.2e-7, 82.8).  The 4-bit instruction rounds (4e-8 over 7,168 elements), its tiles
// stay whole.
#pragma once

#include "kda_few_tc.cuh"

namespace kda {
namespace fewtc {

constexpr int kStayThreads = 384;
constexpr int kMaxExperts = 1024;

// Mx: e2m1, else bf16.  T: columns of a token.
template <int N, int T, bool Mx> struct Stay {
    static constexpr int tokens = N / T;
    static constexpr int stage_k = Mx ? 256 : 64;
    static constexpr int chunk = Mx ? 1 << 30 : 2;               // stages that an accumulator takes
    static constexpr uint32_t stage = kTileA + N * 128;
    static constexpr int stages = N == 128 ? 6 : T == 1 ? (N == 16 ? 5 : N == 32 ? 4 : 3) : N <= 32 ? 5 : 4;
    static constexpr int per_sm = N <= 64 ? 2 : 1;
    static constexpr int nb = N < 32 ? 1 : N / 32, set = nb < 4 ? 4 : nb, group = 16 + 4 * set;
    static constexpr int acc = N < 32 ? 32 : N;                  // columns from one accumulator to the next
    static constexpr int accs = Mx ? 2 : 4;                      // accumulators: bf16 chunks go on while a tile is put away
    static constexpr int scales_at = accs * acc;
    static constexpr int need = scales_at + (Mx ? kSlots * group : 0);
    static constexpr int tmem = need <= 64 ? 64 : need <= 128 ? 128 : need <= 256 ? 256 : 512;
    static_assert(tmem * per_sm <= 512, "tensor memory of an SM");
    static constexpr int words = 128 + 4 * nb;
    static constexpr uint32_t ring = stages * stage;
    static constexpr uint32_t scales = Mx ? 2 * words * 16 : 0;
    static constexpr uint32_t red = tokens * few::kRedPitch * 4;
    static constexpr uint32_t lists = (2 * kMaxExperts + 2) * 2;
    static constexpr uint32_t smem = ring + scales + red + lists + 1024;
    static_assert((smem + 1024 + 512) * per_sm <= 228 * 1024, "shared memory of an SM");
};

struct StayBarriers {
    uint64_t full[6], empty[6], scales_full[kSlots], scales_empty[kSlots], sums[4], free[4];
    uint32_t tmem;
    int failed;
};

struct StayArgs {
    const uint8_t *w_scales, *b_scales;
    int rows, half, K;    // of one expert's matrix; half: rows between a tile's two runs of 64 (64 where they adjoin)
    int tile_rows;        // rows from one tile to the next
    int tiles;            // per expert
    const int* lists;     // experts in use; which; where their places begin; the places' slots
    int E, top, tokens;   // tokens: rows of the columns' tensor / T
};

// The epilogue is called by warps 8 to 11 with a tile's sums in red[token][128 rows]: put(expert, first row of the tile, first
// place, places, red, warp of four).
template <int N, int T, bool Mx, typename Put>
__device__ __forceinline__ void stay(uint8_t* smem, StayBarriers& bar, const Maps& maps, const StayArgs& a, int* d_status, Put put) {
    using S = Stay<N, T, Mx>;
    const int warp = warp_index(), lane = threadIdx.x & 31;
    uint8_t* ring = smem;
    float* red = reinterpret_cast<float*>(smem + S::ring + S::scales);
    uint16_t* which = reinterpret_cast<uint16_t*>(smem + S::ring + S::scales + S::red);
    uint16_t* begin = which + kMaxExperts;
    // The lists come from two kernels back, which has ended; what this CTA has not waited for itself it reads from L2.
    const int experts = __ldcg(a.lists);
    const int items = experts * a.tiles;
    if ((int)blockIdx.x >= items) return;
    for (int i = threadIdx.x; i <= experts; i += kStayThreads) {
        if (i < experts) which[i] = (uint16_t)__ldcg(a.lists + 1 + i);
        begin[i] = (uint16_t)__ldcg(a.lists + 1 + a.E + i);
    }
    if (warp == 2) {
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
        for (int i = 0; i < S::accs; ++i) {
            mbar_init(&bar.sums[i], 1);
            mbar_init(&bar.free[i], 4);
        }
        bar.failed = 0;
        fence_mbar_init();
    }
    fence_before_sync();
    __syncthreads();
    fence_after_sync();
    few::let_next_kernel_begin();

    const uint32_t base = smem_u32(ring), tm = bar.tmem;
    const int blocks = (a.K + S::stage_k - 1) / S::stage_k, groups = (a.K + kGroupK - 1) / kGroupK;
    const int chunks = Mx ? 1 : (blocks + S::chunk - 1) / S::chunk;
    // what every role walks over: tiles of the experts in use, and an expert's tokens by as many as there are columns for
    const auto walk = [&](auto&& step) {
        uint32_t p = 0;
        for (int it = blockIdx.x; it < items; it += gridDim.x) {
            const int at = it / a.tiles, row0 = (it - at * a.tiles) * a.tile_rows, first = begin[at], last = begin[at + 1];
            for (int c0 = first; c0 < last; c0 += S::tokens, ++p)
                if (!step(p, (int)which[at], row0, c0, min(S::tokens, last - c0))) return;
        }
    };
    if (warp == 0 && lane == 0) {
        bool waited = false;
        uint32_t issued = 0;
        walk([&](uint32_t p, int e, int row0, int c0, int) {
            const auto rows = [&](int kb, uint32_t s) {
                const int x = Mx ? kb * 128 : kb * S::stage_k;
                mbar_expect_tx(&bar.full[s], S::stage);
                tma_2d(base + s * S::stage, &maps.w, x, e * a.rows + row0, &bar.full[s]);
                tma_2d(base + s * S::stage + kTileA / 2, &maps.w, x, e * a.rows + row0 + a.half, &bar.full[s]);
            };
            const auto columns = [&](int kb, uint32_t s) {
                tma_2d(base + s * S::stage + kTileA, &maps.b, Mx ? kb * 128 : kb * S::stage_k, c0 * T, &bar.full[s]);
            };
            int kb = 0;
            if (!waited) {  // the first round's weights, then - once they are written - its columns
                const int round = min(blocks, S::stages);
                for (; kb < round; ++kb) rows(kb, kb);
                few::wait_for_kernel_before();
                for (int i = 0; i < round; ++i) columns(i, i);
                waited = true;
                issued = round;
            }
            for (; kb < blocks; ++kb) {
                const uint32_t i = p * blocks + kb, s = i % S::stages;
                if (!mbar_wait(&bar.empty[s], ((i / S::stages) & 1u) ^ 1u)) {
                    bar.failed = 1;
                    // copies still in flight end before the shared memory goes away
                    for (uint32_t j = issued > S::stages ? issued - S::stages : 0; j < issued; ++j) mbar_wait(&bar.full[j % S::stages], (j / S::stages) & 1u);
                    return false;
                }
                rows(kb, s);
                columns(kb, s);
                issued = i + 1;
            }
            return true;
        });
    } else if (warp == 1) {
        const uint64_t rows = desc_sw128(base, 16, 1024), columns = desc_sw128(base + kTileA, 16, 1024);
        few::wait_for_kernel_before();  // its time does not count against a wait's deadline
        walk([&](uint32_t p, int, int, int, int) {
            bool ok = true;
            uint32_t d = 0, turn = p * chunks;
            for (int kb = 0; kb < blocks && ok; ++kb) {
                const uint32_t i = p * blocks + kb, s = i % S::stages, at = s * (S::stage >> 4);
                const int in_chunk = Mx ? kb : kb % S::chunk;
                if (in_chunk == 0) {
                    ok = warp_wait(&bar.free[turn % S::accs], ((turn / S::accs) & 1u) ^ 1u);
                    d = tm + turn % S::accs * S::acc;
                }
                ok = ok && warp_wait(&bar.full[s], (i / S::stages) & 1u);
                const uint32_t gi = p * groups + kb / 2, slot = gi % kSlots, sf = tm + S::scales_at + slot * S::group;
                if (Mx && ok && (kb & 1) == 0) ok = warp_wait(&bar.scales_full[slot], (gi / kSlots) & 1u);
                if (ok) fence_after_sync();
                if (elected()) {
                    if (ok) {
#pragma unroll
                        for (int kk = 0; kk < 4; ++kk) {
                            if constexpr (Mx) {
                                const int set = 2 * (kb & 1) + (kk >> 1);  // of 128 elements
                                mma_mxf4(d, rows + at + 2 * kk, columns + at + 2 * kk, idesc_mxf4(N, 2 * (kk & 1)), sf + 4 * set,
                                         sf + 16 + S::set * set, (kb | kk) != 0);
                            } else {
                                mma_ss(d, rows + at + 2 * kk, columns + at + 2 * kk, idesc_bf16(128, N, false, false), (in_chunk | kk) != 0);
                            }
                        }
                        mma_commit(&bar.empty[s]);
                        if (Mx && ((kb & 1) || kb == blocks - 1)) mma_commit(&bar.scales_empty[slot]);
                    }
                    if (in_chunk == S::chunk - 1 || kb == blocks - 1) mma_commit(&bar.sums[turn % S::accs]);
                }
                __syncwarp();
                if (in_chunk == S::chunk - 1 || kb == blocks - 1) ++turn;
            }
            if (!ok) bar.failed = 1;
            return ok;
        });
    } else if (Mx && warp >= 4 && warp < 8) {
        const int q = warp & 3;
        const uint32_t quadrant = (uint32_t)q * 32 << 16;
        const int64_t pitch = a.K >> 5;
        const int wa = alignment(a.w_scales, pitch), wb = alignment(a.b_scales, pitch);
        constexpr int kAhead = 3;
        const int token = 32 * q + lane;
        uint4* place = reinterpret_cast<uint4*>(smem + S::ring);
        const uint32_t down = 0x03030303u * (lane & 7);
        // The walk as a cursor, so that loads run ahead of it across tiles.
        struct Cursor {
            const uint8_t *ra, *rb;
            int it, c0, g;
        };
        const auto rows_at = [&](Cursor& c) {  // rows past the matrix and tokens past the last are read as those
            const int at = c.it / a.tiles, e = which[at];
            const int r = (c.it - at * a.tiles) * a.tile_rows + (q < 2 ? 0 : a.half - 64) + 32 * q + lane;
            c.ra = a.w_scales + ((int64_t)e * a.rows + min(r, a.rows - 1)) * pitch;
            c.rb = a.b_scales + (int64_t)min(c.c0 + token, a.tokens - 1) * pitch;
        };
        const auto next = [&](Cursor& c) {
            if (c.it >= items || ++c.g < groups) return;  // behind the end there is nothing to look up
            c.g = 0;
            c.c0 += S::tokens;
            if (c.c0 >= begin[c.it / a.tiles + 1]) {
                c.it += gridDim.x;
                if (c.it >= items) return;
                c.c0 = begin[c.it / a.tiles];
            }
            rows_at(c);
        };
        uint4 av[kAhead], bv[kAhead];
        const auto load_a = [&](const Cursor& c, int i) {
            if (c.it < items) av[i] = load_scales(c.ra, c.g * kGroupK, a.K, wa);
        };
        const auto load_b = [&](const Cursor& c, int i) {
            if (c.it < items && token < 4 * S::nb) bv[i] = load_scales(c.rb, c.g * kGroupK, a.K, wb);
        };
        Cursor head;
        head.it = blockIdx.x, head.c0 = begin[blockIdx.x / a.tiles], head.g = 0;
        rows_at(head);
        Cursor ahead = head;
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            load_a(ahead, i);
            next(ahead);
        }
        few::wait_for_kernel_before();
        ahead = head;
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            load_b(ahead, i);
            next(ahead);
        }
        int left = 0;  // groups to bring
        for (int it = blockIdx.x; it < items; it += gridDim.x) {
            const int at = it / a.tiles;
            left += (begin[at + 1] - begin[at] + S::tokens - 1) / S::tokens * groups;
        }
        bool failed = false;  // once a wait ran out none follows, and the walk goes on: the warps meet in barriers
        for (int g0 = 0; g0 < left; g0 += kAhead) {
#pragma unroll
            for (int i = 0; i < kAhead; ++i) {
                const uint32_t gi = g0 + i;
                if ((int)gi >= left) break;
                uint4* here = place + (gi & 1) * S::words;  // of the exchange's two places
                here[32 * q + lane] = av[i];
                if (token < 4 * S::nb) here[128 + token] = bv[i];
                load_a(ahead, i);
                load_b(ahead, i);
                next(ahead);
                scale_warps_sync();
                const uint32_t slot = gi % kSlots, at = tm + quadrant + S::scales_at + slot * S::group;
                if (!failed) {
                    bool ok = true;
                    if (lane == 0) ok = mbar_wait(&bar.scales_empty[slot], ((gi / kSlots) & 1u) ^ 1u);
                    failed = !__shfl_sync(0xffffffffu, ok ? 1 : 0, 0);
                }
                if (failed) continue;
                fence_after_sync();
                {
                    const uint4 r0 = here[lane], r1 = here[32 + lane], r2 = here[64 + lane], r3 = here[96 + lane];
                    const uint32_t w[16] = {r0.x, r1.x, r2.x, r3.x, r0.y, r1.y, r2.y, r3.y, r0.z, r1.z, r2.z, r3.z, r0.w, r1.w, r2.w, r3.w};
                    tmem_st16(at, w);
                }
#pragma unroll
                for (int h = 0; h < S::nb; h += 4) {
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
        if (failed && lane == 0) bar.failed = 1;
    } else if (warp >= 8) {
        const int q = warp & 3;
        const uint32_t quadrant = (uint32_t)q * 32 << 16;
        few::wait_for_kernel_before();  // before anything is written that an earlier kernel may still read
        bool ok = true;                 // once a wait ran out none follows, as above
        walk([&](uint32_t p, int e, int row0, int c0, int n) {
            for (int k = 0; k < chunks; ++k) {
                const uint32_t turn = p * chunks + k;
                if (lane == 0 && ok) ok = mbar_wait(&bar.sums[turn % S::accs], (turn / S::accs) & 1u);
                ok = __shfl_sync(0xffffffffu, ok ? 1 : 0, 0);
                fence_after_sync();
#pragma unroll 1
                for (int c = 0; c < N && ok; c += 16) {
                    uint32_t v[16];
                    tmem_ld16(tm + quadrant + turn % S::accs * S::acc + c, v);
                    tmem_ld_wait();
#pragma unroll
                    for (int i = 0; i < 16; i += T) {
                        float sum = __uint_as_float(v[i + T - 1]);
#pragma unroll
                        for (int j = T - 2; j >= 0; --j) sum += __uint_as_float(v[i + j]);
                        float& to = red[(c + i) / T * few::kRedPitch + 32 * q + lane];
                        to = k ? to + sum : sum;
                    }
                }
                fence_before_sync();
                __syncwarp();
                if (lane == 0) arrive(&bar.free[turn % S::accs]);
            }
            asm volatile("bar.sync 2, 128;" ::: "memory");
            if (ok) put(e, row0, c0, n, red, q);
            asm volatile("bar.sync 2, 128;" ::: "memory");
            return true;
        });
        if (!ok && lane == 0) bar.failed = 1;
    }
    fence_before_sync();
    __syncthreads();
    if (threadIdx.x == 0 && bar.failed) flag_status(d_status, KDA_ERR_TIMEOUT);
    if (warp == 2) tmem_dealloc(tm, S::tmem);
}

}  // namespace fewtc
}  // namespace kda
