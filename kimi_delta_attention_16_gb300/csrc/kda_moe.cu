// kda_moe.cu -- a mixture-of-experts layer for few tokens: router, choice of experts, the experts'
// products, their weighted sum.
//
//   logit[t][e] = x_t . router_e;  score = sigmoid(logit), or the softmax of the chosen logits
//   choice: the `top` experts with the largest score + bias (logits for the softmax), ties to the lower expert
//   w_tj = scale * score / (sum of the chosen scores)
//   y_t = sum_j w_tj W_out[e_j] (silu(g) u),   (g, u) = the halves of W_in[e_j] x_t
//
// Bound by the bytes of the experts that some token chose; each is read once for all its tokens.  Six launches, each beside
// the end of the one in front: scores, choice with the lists of every expert's tokens, the tokens' columns, first products
// with their activation, second products, sum over a token's experts in the order of their rank (integer codes: the
// columns first).  e2m1 and bf16 experts
// go through the tensor cores (kda_moe_tc.cuh), integer codes through kda_few.cuh.
//
// e2m1, 32 tokens, 8 of 256 experts, 7,168 x 2,048: 597 to 640 us (6.0 to 6.4 TB/s of what has to be read; scores 25, choice
// and columns 12, products 575); one token, 16 of 896, 3,584 x 2,048: 56 us, half of it the chain of launches; bf16, 4 tokens, 6
// of 64, 2,048 x 1,408: 74 to 81 us (4.5 to 4.9 TB/s).  Meant for few tokens: an expert's weights pass once per 16 of its tokens (e2m1, 8 of
// 256, 3,584 x 2,048: 1,024 tokens 2.0 ms, 4,096 tokens 7.9 ms).
#include "kda_few.cuh"
#include "kda_moe_tc.cuh"
#include "kda_serve.cuh"
#include "kda_wide.cuh"

namespace kda {

namespace {

using namespace few;

// ------------------------------------------------------------------ scores
// A choice between two experts hangs on the last digits of a sum over thousands of products, so logits and scores are
// pairs of fp32 (kda_wide.cuh).  A block takes one expert and TB tokens, its warps share the rows.  One token: all of the
// router is on its way at once; a block that stands for four takes 6 us longer (896 experts, 3,584 channels).  More: four
// tokens share what is read of the router, 99 us instead of 118 for a small layer behind the same router and 32
// tokens; four experts by four tokens: 97.
constexpr int kScoreThreads = 256, kScoreWarps = 8;

__device__ __forceinline__ uint32_t ordered(float v) {  // a larger value is a larger integer
    const uint32_t b = __float_as_uint(v + 0.0f);
    return b >> 31 ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ uint64_t ordered(Wide v) {  // NaN is the smallest
    return isnan(v.hi) ? 0 : (uint64_t)ordered(v.hi) << 32 | ordered(v.lo);
}

template <typename T> __device__ __forceinline__ void load8_any(const T* p, bool aligned, float (&v)[8]) {
    if (aligned) {
        load8(p, v);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = to_f(p[i]);
    }
}

template <typename Tr, int TB>
__global__ void __launch_bounds__(kScoreThreads) k_moe_scores(const bf16* __restrict__ x, int64_t xs, bool xwide, const Tr* __restrict__ router,
                                                              bool rwide, const float* __restrict__ bias, int M, int E, int D,
                                                              int sigmoid, Wide* __restrict__ logits, uint64_t* __restrict__ key,
                                                              int* __restrict__ done) {
    __shared__ Wide sums[kScoreWarps][TB];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int e = blockIdx.x, t0 = blockIdx.y * TB;
    if (e == 0 && t0 == 0 && threadIdx.x == 0) *done = 0;
    Sum2 s[TB];
#pragma unroll TB == 1 ? 2 : 1
    for (int k = threadIdx.x * 8; k < D; k += kScoreThreads * 8) {
        float rv[8], xv[TB][8];
        load8_any(router + (int64_t)e * D + k, rwide, rv);
#pragma unroll
        for (int j = 0; j < TB; ++j) load8_any(x + (int64_t)min(t0 + j, M - 1) * xs + k, xwide, xv[j]);
#pragma unroll
        for (int j = 0; j < TB; ++j)
#pragma unroll
            for (int v = 0; v < 8; ++v) {
                const float p = xv[j][v] * rv[v];  // exact for a bf16 router
                s[j].add(p);
                if constexpr (sizeof(Tr) == 4) s[j].lo += fmaf(xv[j][v], rv[v], -p);
            }
    }
#pragma unroll
    for (int j = 0; j < TB; ++j) {
#pragma unroll
        for (int d = 16; d; d >>= 1) {
            const float h = __shfl_xor_sync(0xffffffffu, s[j].hi, d), l = __shfl_xor_sync(0xffffffffu, s[j].lo, d);
            s[j].add(h);
            s[j].lo += l;
        }
        if (lane == 0) sums[warp][j] = wide(s[j]);
    }
    __syncthreads();
    const int j = threadIdx.x;
    let_next_kernel_begin();
    wait_for_kernel_before();  // the columns' kernel, if one runs beside this: what comes next counts on both
    if (j < TB && t0 + j < M) {
        Wide v = sums[0][j];
#pragma unroll
        for (int w = 1; w < kScoreWarps; ++w) v = add(v, sums[w][j]);
        const int64_t at = (int64_t)(t0 + j) * E + e;
        const Wide logit = v;
        // next to 1/2 the score is 1/2 + logit / 4 (what follows is below 2^-59), which loses no digits of the logit's
        constexpr float kSmall = 0x1p-18f;
        if (sigmoid) v = fabsf(logit.hi) < kSmall ? add(Wide{0.5f, 0.f}, Wide{0.25f * logit.hi, 0.25f * logit.lo}) : sigmoid_wide(v);
        logits[at] = logit;
        // scores next to 1 and to 1/2 are equal where fp64 holds them equal; those well below 1/2 without a bias are ordered by their
        // logits (negative, so below every other score), which do not underflow
        key[at] = ordered(!sigmoid ? logit : bias ? to_53_bits(add(v, Wide{bias[e], 0.f})) : logit.hi <= -kSmall ? logit : to_53_bits(v));
    }
}

// ------------------------------------------------------------------ choice and lists
constexpr int kPickThreads = 512, kPickWarps = 16;

// The largest key of the warp and the lowest index among its holders; a lane without a key has index 0x7fffffff.
__device__ __forceinline__ int largest(uint64_t key, int index, uint64_t& top) {
    const bool has = index != 0x7fffffff;
    const uint32_t hi = __reduce_max_sync(0xffffffffu, has ? (uint32_t)(key >> 32) : 0u);
    const bool in = has && (uint32_t)(key >> 32) == hi;
    const uint32_t lo = __reduce_max_sync(0xffffffffu, in ? (uint32_t)key : 0u);
    top = (uint64_t)hi << 32 | lo;
    return (int)__reduce_min_sync(0xffffffffu, in && (uint32_t)key == lo ? (uint32_t)index : 0x7fffffffu);
}

// A block per token: each warp orders the best `top` of its 64 experts, one warp merges the sixteen lists.  The block
// that finishes last lists the slots (token, rank) by expert; the order of an expert's slots is free, since every
// column of a product is computed alike.
__global__ void __launch_bounds__(kPickThreads) k_moe_pick(const Wide* __restrict__ logits, const uint64_t* __restrict__ key, int M, int E, int top,
                                                           int sigmoid, float scale, int* __restrict__ ids, float* __restrict__ weights,
                                                           int* __restrict__ done, int* __restrict__ lists, int* __restrict__ user_ids,
                                                           float* __restrict__ user_weights) {
    __shared__ uint64_t best_key[kPickWarps][33];
    __shared__ int best_id[kPickWarps][33];
    __shared__ int count[1024], begin[1024];
    __shared__ uint32_t warp_sum[kPickWarps];
    __shared__ bool last;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, t = blockIdx.x;
    wait_for_kernel_before();
    let_next_kernel_begin();
    {
        // a warp's experts are 64 in a row, two per lane
        uint64_t k[2];
        int id[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int e = warp * 64 + 32 * i + lane;
            k[i] = e < E ? key[(int64_t)t * E + e] : 0;
            id[i] = e < E ? e : 0x7fffffff;
        }
        if (id[1] != 0x7fffffff && k[1] > k[0]) {  // the better one first; the lower index where they are equal
            const uint64_t kk = k[0];
            const int ii = id[0];
            k[0] = k[1], id[0] = id[1], k[1] = kk, id[1] = ii;
        }
        int mine = 0x7fffffff;
        uint64_t mine_key = 0;
        for (int j = 0; j < top; ++j) {
            uint64_t v;
            const int e = largest(k[0], id[0], v);
            if (lane == j) mine = e, mine_key = v;
            if (id[0] == e) k[0] = k[1], id[0] = id[1], k[1] = 0, id[1] = 0x7fffffff;
        }
        best_key[warp][lane] = mine_key;
        best_id[warp][lane] = mine;
        if (lane == 0) best_id[warp][32] = 0x7fffffff;
    }
    __syncthreads();
    if (warp == 0) {
        int head = 0, mine = 0;
        uint64_t k = lane < kPickWarps ? best_key[lane][0] : 0, v;
        int id = lane < kPickWarps ? best_id[lane][0] : 0x7fffffff;
        for (int j = 0; j < top; ++j) {
            const int e = largest(k, id, v);
            if (lane == j) mine = e;
            if (id == e) {
                ++head;
                k = best_key[lane][head];
                id = best_id[lane][head];
            }
        }
        // Weights are quotients: every score times e^-m is as good, and does not underflow with m the largest logit, or 0
        // for sigmoids where that is positive.
        Wide w;
        if (lane < top) w = logits[(int64_t)t * E + mine];
        float m = lane < top ? w.hi : -INFINITY;
#pragma unroll
        for (int d = 16; d; d >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));  // leaves NaN out
        const Wide first = from(0xffffffffu, w, 0);  // the largest logit itself, for the softmax
        if (lane < top) {
            if (!sigmoid)
                w = exp_wide(add(w, minus(first)));
            else if (w.hi > 0.f)
                w = sigmoid_wide(w);
            else if (!isnan(w.hi))
                w = over(exp_wide(add(w, Wide{-fminf(m, 0.f), 0.f})), add(Wide{1.f, 0.f}, exp_wide(w)));
        }
        Wide sum = w;
#pragma unroll
        for (int d = 16; d; d >>= 1) sum = add(sum, Wide{__shfl_xor_sync(0xffffffffu, sum.hi, d), __shfl_xor_sync(0xffffffffu, sum.lo, d)});
        if (lane < top) {
            const Wide q = times(over(w, sum), Wide{scale, 0.f});
            const int slot = t * top + lane;
            ids[slot] = mine;
            weights[slot] = q.hi;
            if (user_ids) user_ids[slot] = mine;
            if (user_weights) user_weights[slot] = q.hi;
        }
        __syncwarp();
        if (lane == 0) {
            __threadfence();
            last = atomicAdd(done, 1) == M - 1;
        }
    }
    __syncthreads();
    if (!last) return;
    __threadfence();
    for (int i = threadIdx.x; i < 1024; i += kPickThreads) count[i] = 0;
    __syncthreads();
    const int slots = M * top;
    for (int i = threadIdx.x; i < slots; i += kPickThreads) atomicAdd(&count[__ldcg(ids + i)], 1);
    __syncthreads();
    // running sums over the experts: slots in the low 20 bits, experts in use above them
    const int c0 = count[2 * threadIdx.x], c1 = count[2 * threadIdx.x + 1];
    const uint32_t own0 = (uint32_t)c0 | (c0 ? 1u << 20 : 0u), own1 = (uint32_t)c1 | (c1 ? 1u << 20 : 0u);
    uint32_t run = own0 + own1;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const uint32_t o = __shfl_up_sync(0xffffffffu, run, d);
        if (lane >= d) run += o;
    }
    if (lane == 31) warp_sum[warp] = run;
    __syncthreads();
    uint32_t before = run - own0 - own1;
    for (int w = 0; w < warp; ++w) before += warp_sum[w];
    int* which = lists + 1;
    int* starts = lists + 1 + E;
    int* listed = lists + 2 + 2 * E;
    constexpr uint32_t kLow = (1u << 20) - 1;
    begin[2 * threadIdx.x] = before & kLow;
    begin[2 * threadIdx.x + 1] = (before & kLow) + c0;
    if (c0) {
        which[before >> 20] = 2 * threadIdx.x;
        starts[before >> 20] = before & kLow;
    }
    before += own0;
    if (c1) {
        which[before >> 20] = 2 * threadIdx.x + 1;
        starts[before >> 20] = before & kLow;
    }
    before += own1;
    if (threadIdx.x == kPickThreads - 1) {
        lists[0] = before >> 20;
        starts[before >> 20] = before & kLow;
    }
    __syncthreads();
    for (int i = threadIdx.x; i < slots; i += kPickThreads) listed[atomicAdd(&begin[__ldcg(ids + i)], 1)] = i;
}

// ------------------------------------------------------------------ experts in integer codes
constexpr int kExpertWarps = 8;

struct Experts {
    Weights w;                 // of expert 0
    int64_t w_bytes, s_bytes;  // of one expert
    Columns x;
    int rows, K, group;        // of one expert's matrix
    const int* lists;
    int E, top;
    __device__ __forceinline__ Weights matrix(int e) const { return Weights{w.codes + e * w_bytes, w.scales + e * s_bytes}; }
};

struct Direct {  // the operands as they were given, for sums that come out as NaN or infinite
    const uint8_t *codes, *scales;
    const bf16* x;
    int64_t xs;
    // Slots with this weight need no such sum: a token whose logits are NaN has a y of NaN whatever its hidden values.  Its experts
    // are the lowest ones, for all such tokens (1,000 of 2,000 tokens, 4 of 16 experts of 1,024 x 256: 41 ms, integer codes 150,
    // with the sums, 1.1 and 1.6 without, 0.6 and 0.7 for ordinary tokens).
    const float* weights;
    __device__ __forceinline__ bool wanted(int slot) const { return !isnan(weights[slot]); }
};

// First products.  Warps 0 to 3 take 128 rows of the gate's half, 4 to 7 the same of the other; the hidden values become
// two columns of the second products' (value and remainder) where they arise, 128 rows under one power of two.
template <int NT, int GS, int SB>
__global__ void __launch_bounds__(32 * kExpertWarps, 1) k_moe_in(const Experts p, const Direct given, const Columns hidden) {
    using L = Layout<kExpertWarps, NT, GS, SB>;
    constexpr int kPitch = 256 + 4;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ int of[L::cols];
    float* sums = reinterpret_cast<float*>(smem + L::bytes);  // [cols][256 rows]
    wait_for_kernel_before();
    let_next_kernel_begin();
    if ((int)blockIdx.y >= p.lists[0]) return;
    const int e = p.lists[1 + blockIdx.y], first = p.lists[1 + p.E + blockIdx.y], last = p.lists[2 + p.E + blockIdx.y];
    const int* slots = p.lists + 2 + 2 * p.E;
    const int row0 = blockIdx.x * 128, F = p.rows / 2, warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const int runs = (F + kRun - 1) / kRun;
    const auto row_of = [&](int, int tile, int r) -> int64_t { return min(row0 + few::kRows * (tile & 3) + r, F - 1) + (tile >= 4 ? F : 0); };
    const Weights m = p.matrix(e);
    for (int c0 = first; c0 < last; c0 += L::cols) {
        const int n = min(L::cols, last - c0);
        __syncthreads();
        if (threadIdx.x < n) of[threadIdx.x] = slots[c0 + threadIdx.x] / p.top;
        __syncthreads();
        products<L>(smem, m, p.x, p.K, of, n, 1, 1, row_of, [&](int, const float (&acc)[2][NT][4]) {
#pragma unroll
            for (int u = 0; u < 2; ++u)
#pragma unroll
                for (int c = 0; c < NT; ++c)
#pragma unroll
                    for (int j = 0; j < 4; ++j) sums[(8 * c + 2 * t + (j & 1)) * kPitch + few::kRows * warp + 16 * u + g + 8 * (j >> 1)] = acc[u][c][j];
        });
        __syncthreads();
        __half* columns = const_cast<__half*>(hidden.x);
        float *factor = const_cast<float*>(hidden.factor), *group_sums = const_cast<float*>(hidden.sums);
        const int out_groups = F / p.group;
        // a warp per token: four values a lane, rows 32 i + lane
        for (int c = warp; c < n; c += kExpertWarps) {
            float v[4];
            uint32_t top = 0;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                float gate = sums[c * kPitch + 32 * i + lane], up = sums[c * kPitch + 128 + 32 * i + lane];
                if (row0 + 32 * i + lane < F && !(isfinite(gate) && isfinite(up)) && given.wanted(slots[c0 + c])) {
                    const bf16* x = given.x + of[c] * given.xs;
                    const int64_t rg = row0 + 32 * i + lane, ru = rg + F;
                    const int row_scales = p.K / p.group * SB;
                    gate = few::direct(m.codes + rg * (p.K / 2), m.scales + rg * row_scales, SB, p.group, x, p.K);
                    up = few::direct(m.codes + ru * (p.K / 2), m.scales + ru * row_scales, SB, p.group, x, p.K);
                }
                v[i] = row0 + 32 * i + lane < F ? gate / (1.0f + expf(-gate)) * up : 0.f;
                top = max(top, __float_as_uint(v[i]) & 0x7fffffffu);
            }
            top = __reduce_max_sync(0xffffffffu, top);
            float up, down;
            run_scale(top >> 23, up, down);
            // element k of eight lies at the place where codes come out of a word: (0,4) (1,5) (2,6) (3,7)
            const int place = (lane & ~7) + 2 * (lane & 3) + (lane >> 2 & 1);
            const int64_t at = (int64_t)(c0 + c) * 2;
            float sum_hi = 0.f, sum_lo = 0.f;  // of a group, as far as it goes
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if (row0 + 32 * i >= F) break;  // F is a multiple of the group
                const float x = v[i] * up;
                const __half hi = __float2half_rn(x);
                const float h = __half2float(hi);
                const __half lo = __float2half_rn(isinf(h) ? 0.f : x - h);
                columns[at * F + row0 + 32 * i + place] = hi;
                columns[(at + 1) * F + row0 + 32 * i + place] = lo;
                sum_hi += h, sum_lo += __half2float(lo);
                if ((i + 1) * 32 % p.group == 0) {
#pragma unroll
                    for (int d = 16; d; d >>= 1) {
                        sum_hi += __shfl_xor_sync(0xffffffffu, sum_hi, d);
                        sum_lo += __shfl_xor_sync(0xffffffffu, sum_lo, d);
                    }
                    const int group = (row0 + 32 * i) / p.group;
                    if (lane < 2) group_sums[(at + lane) * out_groups + group] = kSumOf * (lane ? sum_lo : sum_hi);
                    sum_hi = sum_lo = 0.f;
                }
            }
            if (lane < 2) factor[(at + lane) * runs + blockIdx.x] = down;
        }
    }
}

// Second products: parts[slot][d] = w_slot W_out hidden_slot, from two columns a slot.
template <int NT, int GS, int SB>
__global__ void __launch_bounds__(32 * kExpertWarps, 1) k_moe_out(const Experts p, const float* __restrict__ weights, float* __restrict__ parts) {
    using L = Layout<kExpertWarps, NT, GS, SB>;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ int of[L::cols];
    wait_for_kernel_before();
    let_next_kernel_begin();
    if ((int)blockIdx.y >= p.lists[0]) return;
    const int e = p.lists[1 + blockIdx.y], first = p.lists[1 + p.E + blockIdx.y], last = p.lists[2 + p.E + blockIdx.y];
    const int* slots = p.lists + 2 + 2 * p.E;
    const int row0 = blockIdx.x * 256, warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const auto row_of = [&](int, int tile, int r) -> int64_t { return row0 + few::kRows * tile < p.rows ? min(row0 + few::kRows * tile + r, p.rows - 1) : -1; };
    const Weights m = p.matrix(e);
    for (int c0 = first; c0 < last; c0 += L::cols / 2) {
        const int n = min(L::cols / 2, last - c0);
        __syncthreads();
        if (threadIdx.x < 2 * n) of[threadIdx.x] = 2 * c0 + threadIdx.x;
        __syncthreads();
        products<L>(smem, m, p.x, p.K, of, 2 * n, 1, 1, row_of, [&](int, const float (&acc)[2][NT][4]) {
#pragma unroll
            for (int c = 0; c < NT; ++c) {
                const int token = 4 * c + t;  // columns 8 c + 2 t and the next
                if (token >= n) continue;
                const int slot = slots[c0 + token];
                const float w = weights[slot];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int row = row0 + few::kRows * warp + g + 8 * j;
                    const float(&s)[4] = acc[j >> 1][c];
                    if (row >= p.rows) continue;
                    float v = s[2 * (j & 1)] + s[2 * (j & 1) + 1];
                    if (!isfinite(v) && !isnan(w)) {
                        const int64_t at = 2 * (int64_t)(c0 + token);
                        v = few::direct_columns(m.codes + (int64_t)row * (p.K / 2), m.scales + (int64_t)row * (p.K / p.group) * SB, SB, p.group,
                                                p.x.x + at * p.K, p.x.x + (at + 1) * p.K, p.x.factor + at * ((p.K + kRun - 1) / kRun), p.K);
                    }
                    parts[(int64_t)slot * p.rows + row] = w * v;
                }
            }
        });
    }
}

// ------------------------------------------------------------------ e2m1 and bf16 experts
// The place of a slot in the lists is its row in the columns of both products: a token's columns are repeated for each of
// its experts.  (Tokens' own columns for all experts at once, where they fit: the same time for 1 to 16 tokens.)
//
// A kernel may begin beside the one in front of it.  That one, the columns' or the first products', has waited for the
// choice before it let this one begin, so the lists are complete, and weights and their scales can be on their way
// before the columns are written.
// First products: the hidden values become digits (four bf16 columns, the last of zeros, for bf16 weights) where they
// arise.  32 rows of a token share a scale: a warp's lanes.
template <int N, bool Mx>
__global__ void __launch_bounds__(fewtc::kStayThreads, fewtc::Stay<N, Mx ? 8 : 1, Mx>::per_sm)
k_moe_in_tc(const __grid_constant__ fewtc::Maps maps, const fewtc::StayArgs p, const Direct given, void* __restrict__ columns,
            uint8_t* __restrict__ scales, int* d_status) {
    extern __shared__ uint8_t smem_raw[];
    __shared__ fewtc::StayBarriers bar;
    const uint32_t raw = tc::smem_u32(smem_raw);
    uint8_t* smem = smem_raw + (((raw + 1023u) & ~1023u) - raw);
    const int lane = threadIdx.x & 31, F = p.half;
    const int* slots = p.lists + 2 + 2 * p.E;
    fewtc::stay<N, Mx ? 8 : 1, Mx>(smem, bar, maps, p, d_status, [&](int e, int row0, int c0, int n, const float* red, int q) {
        for (int i = q; i < 2 * n; i += 4) {
            const int c = i >> 1, r = (i & 1) * 32 + lane, f = row0 + r, token = slots[c0 + c] / p.top;
            const float* sum = red + c * kRedPitch + r;
            float gate = sum[0], up = sum[64];
            if constexpr (Mx) {
                if (f < F && !(isfinite(gate) && isfinite(up)) && given.wanted(slots[c0 + c])) {
                    const bf16* row = given.x + (int64_t)token * given.xs;
                    const int64_t g = (int64_t)e * p.rows + f, u = g + F;
                    gate = fewtc::direct(given.codes + g * (p.K / 2), given.scales + g * (p.K / 32), row, p.K);
                    up = fewtc::direct(given.codes + u * (p.K / 2), given.scales + u * (p.K / 32), row, p.K);
                }
            }
            float v = f < F ? gate / (1.0f + expf(-gate)) * up : 0.f;
            if constexpr (Mx) {
                const uint32_t top = __reduce_max_sync(0xffffffffu, __float_as_uint(v) & 0x7fffffffu);
                fewtc::put_digits_of_lanes(v, top, f < F, c0 + c, f, F, static_cast<uint8_t*>(columns), scales);
            } else if (f < F) {
                bf16* to = static_cast<bf16*>(columns) + (int64_t)(c0 + c) * 4 * F + f;
#pragma unroll
                for (int t = 0; t < 3; ++t) {
                    const bf16 h = __float2bfloat16_rn(v);
                    to[(int64_t)t * F] = h;
                    v = isfinite(__bfloat162float(h)) ? v - __bfloat162float(h) : 0.f;
                }
                to[(int64_t)3 * F] = __float2bfloat16_rn(0.f);
            }
        }
    });
}

// Second products: parts[slot][d] = w_slot W_out hidden_slot.
template <int N, bool Mx>
__global__ void __launch_bounds__(fewtc::kStayThreads, fewtc::Stay<N, Mx ? 8 : 4, Mx>::per_sm)
k_moe_out_tc(const __grid_constant__ fewtc::Maps maps, const fewtc::StayArgs p, const float* __restrict__ weights, float* __restrict__ parts,
             int* d_status) {
    extern __shared__ uint8_t smem_raw[];
    __shared__ fewtc::StayBarriers bar;
    const uint32_t raw = tc::smem_u32(smem_raw);
    uint8_t* smem = smem_raw + (((raw + 1023u) & ~1023u) - raw);
    const int* slots = p.lists + 2 + 2 * p.E;
    fewtc::stay<N, Mx ? 8 : 4, Mx>(smem, bar, maps, p, d_status, [&](int, int row0, int c0, int n, const float* red, int q) {
        for (int i = q * 32 + (threadIdx.x & 31); i < n * 32; i += 128) {
            const int c = i >> 5, r = (i & 31) * 4;
            if (row0 + r >= p.rows) continue;  // rows are a multiple of 8
            float4 v = *reinterpret_cast<const float4*>(red + c * kRedPitch + r);
            const int slot = slots[c0 + c];
            const float w = weights[slot];
            v.x *= w, v.y *= w, v.z *= w, v.w *= w;
            *reinterpret_cast<float4*>(parts + (int64_t)slot * p.rows + row0 + r) = v;
        }
    });
}

// y[t][d] = the sum of the token's parts, in the order of their rank.
template <typename T>
__global__ void __launch_bounds__(256) k_moe_sum(const float* __restrict__ parts, int M, int D, int top, T* __restrict__ y, int64_t ys) {
    const int t = blockIdx.y;
    wait_for_kernel_before();
    for (int d = (blockIdx.x * 256 + threadIdx.x) * 4; d < D; d += gridDim.x * 1024) {  // D is a multiple of 8
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
        for (int j = 0; j < top; ++j) {
            const float4 p = *reinterpret_cast<const float4*>(parts + (int64_t)(t * top + j) * D + d);
            v.x += p.x, v.y += p.y, v.z += p.z, v.w += p.w;
        }
        T* o = y + (int64_t)t * ys + d;
        o[0] = from_f<T>(v.x), o[1] = from_f<T>(v.y), o[2] = from_f<T>(v.z), o[3] = from_f<T>(v.w);
    }
}

// ------------------------------------------------------------------ launches
template <typename Tr> cudaError_t launch_scores(const kda_moe_args& a, int64_t xs, bool xwide, Wide* logits, uint64_t* key, int* done, bool beside,
                                               cudaStream_t s) {
    const bf16* x = static_cast<const bf16*>(a.x);
    const Tr* r = static_cast<const Tr*>(a.router);
    const bool rwide = reinterpret_cast<uintptr_t>(r) % 16 == 0;
    const int sg = a.score == KDA_SCORE_SIGMOID;
    const auto go = [&](auto kernel, int tb) {
        return launch_kernel(kernel, dim3(a.E, (a.M + tb - 1) / tb), kScoreThreads, 1, 0, beside, s, x, xs, xwide, r, rwide, a.bias, a.M,
                             a.E, a.D, sg, logits, key, done);
    };
    return a.M == 1 ? go(k_moe_scores<Tr, 1>, 1) : go(k_moe_scores<Tr, 4>, 4);
}

template <int NT, int GS, int SB>
cudaError_t launch_experts(const kda_moe_args& a, const Experts& in, const Experts& out, const Direct& given, const float* weights, float* parts,
                           int most, cudaStream_t s) {
    using L = Layout<kExpertWarps, NT, GS, SB>;
    constexpr int kSums = L::cols * (256 + 4) * 4;
    static_assert(L::bytes + kSums <= 227 * 1024, "shared memory of an SM");
    const cudaError_t e = launch_kernel(k_moe_in<NT, GS, SB>, dim3((a.F + 127) / 128, most), L::threads, 1, L::bytes + kSums, true, s, in, given, out.x);
    if (e) return e;
    return launch_kernel(k_moe_out<NT, GS, SB>, dim3((a.D + 255) / 256, most), L::threads, 1, L::bytes, true, s, out, weights, parts);
}

template <int N, bool Mx>
cudaError_t launch_in_tc(const fewtc::Maps& maps, const fewtc::StayArgs& p, int most, const Direct& given, void* columns, uint8_t* scales, int* d_status,
                         cudaStream_t s) {
    using S = fewtc::Stay<N, Mx ? 8 : 1, Mx>;
    const int64_t items = (int64_t)most * p.tiles;
    return launch_kernel(k_moe_in_tc<N, Mx>, dim3(items < 152 * S::per_sm ? items : 152 * S::per_sm), fewtc::kStayThreads, 1, S::smem, true, s, maps, p,
                         given, columns, scales, d_status);
}
template <int N, bool Mx>
cudaError_t launch_out_tc(const fewtc::Maps& maps, const fewtc::StayArgs& p, int most, const float* weights, float* parts, int* d_status, cudaStream_t s) {
    using S = fewtc::Stay<N, Mx ? 8 : 4, Mx>;
    const int64_t items = (int64_t)most * p.tiles;
    return launch_kernel(k_moe_out_tc<N, Mx>, dim3(items < 152 * S::per_sm ? items : 152 * S::per_sm), fewtc::kStayThreads, 1, S::smem, true, s, maps, p,
                         weights, parts, d_status);
}

// Columns that a pass over an expert's tile holds: for `tokens` tokens of T columns each, 16 to 128.
int box_for(int tokens, int T, int most) {
    int box = 16;
    while (box < most && box / T < tokens) box *= 2;
    return box;
}

template <bool Mx>
cudaError_t launch_experts_tc(const kda_moe_args& a, const MoePlan& p, const int* lists, const bf16* x, int64_t xs, bool xwide, const float* weights,
                              float* parts, int most, int columns, cudaStream_t s) {
    char* ws = static_cast<char*>(a.workspace);
    const int slots = a.M * a.top;
    uint8_t* xc = reinterpret_cast<uint8_t*>(ws + p.x_columns);
    uint8_t* hc = reinterpret_cast<uint8_t*>(ws + p.hidden);
    uint8_t *xsc = xc + fewtc::digits_bytes(slots, a.D), *hsc = hc + fewtc::digits_bytes(slots, a.F);
    const int in_box = box_for(columns, Mx ? 8 : 1, Mx ? 128 : 64), out_box = box_for(columns, Mx ? 8 : 4, Mx ? 128 : 64);
    const int* of = lists + 2 + 2 * a.E;
    fewtc::Maps in, out;
    cudaError_t e = cudaSuccess;
    if constexpr (Mx) {
        if (!fewtc::encode_maps(&in, a.w_in, (int64_t)a.E * 2 * a.F, xc, slots, a.D, in_box) ||
            !fewtc::encode_maps(&out, a.w_out, (int64_t)a.E * a.D, hc, slots, a.F, out_box))
            return cudaErrorInvalidValue;
        e = fewtc::launch_digits(x, xs, xwide, of, a.top, slots, a.D, xc, xsc, s);
    } else {
        if (!fewtc::encode_maps_bf16(&in, a.w_in, (int64_t)a.E * 2 * a.F, xc, slots, a.D, in_box) ||
            !fewtc::encode_maps_bf16(&out, a.w_out, (int64_t)a.E * a.D, hc, 4 * (int64_t)slots, a.F, out_box))
            return cudaErrorInvalidValue;
        e = fewtc::launch_rows(x, xs, xwide, of, a.top, slots, a.D, reinterpret_cast<bf16*>(xc), s);
    }
    if (e) return e;
    fewtc::StayArgs pi = {}, po = {};
    pi.w_scales = static_cast<const uint8_t*>(a.w_in_scales), pi.b_scales = xsc;
    pi.rows = 2 * a.F, pi.half = a.F, pi.K = a.D, pi.tile_rows = kTileRows / 2, pi.tiles = (a.F + 63) / 64;
    pi.lists = lists, pi.E = a.E, pi.top = a.top, pi.tokens = slots;
    po = pi;
    po.w_scales = static_cast<const uint8_t*>(a.w_out_scales), po.b_scales = hsc;
    po.rows = a.D, po.half = 64, po.K = a.F, po.tile_rows = kTileRows, po.tiles = (a.D + kTileRows - 1) / kTileRows;
    const Direct given{static_cast<const uint8_t*>(a.w_in), static_cast<const uint8_t*>(a.w_in_scales), x, xs, weights};
    switch (in_box) {
        case 16: e = launch_in_tc<16, Mx>(in, pi, most, given, hc, hsc, a.d_status, s); break;
        case 32: e = launch_in_tc<32, Mx>(in, pi, most, given, hc, hsc, a.d_status, s); break;
        case 64: e = launch_in_tc<64, Mx>(in, pi, most, given, hc, hsc, a.d_status, s); break;
        default:
            if constexpr (Mx) e = launch_in_tc<128, Mx>(in, pi, most, given, hc, hsc, a.d_status, s);
    }
    if (e) return e;
    switch (out_box) {
        case 16: return launch_out_tc<16, Mx>(out, po, most, weights, parts, a.d_status, s);
        case 32: return launch_out_tc<32, Mx>(out, po, most, weights, parts, a.d_status, s);
        case 64: return launch_out_tc<64, Mx>(out, po, most, weights, parts, a.d_status, s);
        default:
            if constexpr (Mx) return launch_out_tc<128, Mx>(out, po, most, weights, parts, a.d_status, s);
            return cudaErrorInvalidValue;  // not reached: bf16 boxes end at 64
    }
}

template <int NT, int SB, typename... A> cudaError_t launch_group(int group, A&&... args) {
    return group == 32   ? launch_experts<NT, 8, SB>(std::forward<A>(args)...)
           : group == 64 ? launch_experts<NT, 4, SB>(std::forward<A>(args)...)
                         : launch_experts<NT, 2, SB>(std::forward<A>(args)...);
}
template <int NT, typename... A> cudaError_t launch_codes(bool bf16_scales, A&&... args) {
    return bf16_scales ? launch_group<NT, 2>(std::forward<A>(args)...) : launch_group<NT, 4>(std::forward<A>(args)...);
}

}  // namespace

MoePlan moe_plan(const kda_moe_args& a) {
    MoePlan p;
    size_t at = 0;
    const size_t slots = (size_t)a.M * a.top;
    auto take = [&](size_t bytes) {
        const size_t here = at;
        at = (at + bytes + 255) / 256 * 256;
        return here;
    };
    p.logits = take((size_t)a.M * a.E * 8);
    p.key = take((size_t)a.M * a.E * 8);
    p.done = take(4);
    p.ids = take(slots * 4);
    p.weights = take(slots * 4);
    p.lists = take((2 + 2 * (size_t)a.E + slots) * 4);
    const bool mx = a.format == KDA_WEIGHT_E2M1, tc = mx || a.format == KDA_WEIGHT_BF16;
    p.x_columns = take(mx ? fewtc::digits_bytes(slots, a.D) + fewtc::digit_scales_bytes(slots, a.D) : tc ? slots * a.D * 2 : few::columns_bytes(a.M, a.D, a.group));
    p.hidden = take(mx ? fewtc::digits_bytes(slots, a.F) + fewtc::digit_scales_bytes(slots, a.F) : tc ? slots * a.F * 8 : few::columns_bytes(2 * slots, a.F, a.group));
    p.parts = take(slots * a.D * 4);
    p.workspace = at;
    return p;
}

cudaError_t launch_moe(const kda_moe_args& a, const MoePlan& p, cudaStream_t s) {
    char* ws = static_cast<char*>(a.workspace);
    Wide* logits = reinterpret_cast<Wide*>(ws + p.logits);
    uint64_t* key = reinterpret_cast<uint64_t*>(ws + p.key);
    int* ids = reinterpret_cast<int*>(ws + p.ids);
    float* weights = reinterpret_cast<float*>(ws + p.weights);
    int* lists = reinterpret_cast<int*>(ws + p.lists);
    float* parts = reinterpret_cast<float*>(ws + p.parts);
    const int64_t xs = a.x_stride ? a.x_stride : a.D, ys = a.y_stride ? a.y_stride : a.D;
    const bool xwide = reinterpret_cast<uintptr_t>(a.x) % 16 == 0 && (xs % 8 == 0 || a.M == 1);
    int* done = reinterpret_cast<int*>(ws + p.done);
    // columns for twice an expert's even share of the slots, and no more than there are tokens
    const int slots = a.M * a.top, most = slots < a.E ? slots : a.E;
    const int even = 2 * ((slots + a.E - 1) / a.E) + 2, columns = a.M < even ? a.M : even;
    const bf16* x = static_cast<const bf16*>(a.x);
    const bool mx = a.format == KDA_WEIGHT_E2M1, tc = mx || a.format == KDA_WEIGHT_BF16;
    cudaError_t e;
    // integer codes: columns that need no lists come first, the router's scores run beside them
    if (!tc) {
        e = launch_halves(x, xs, xwide, a.M, a.D, a.group, columns_at(ws + p.x_columns, a.M, a.D), s);
        if (e) return e;
    }
    e = a.router_dtype == KDA_BF16 ? launch_scores<bf16>(a, xs, xwide, logits, key, done, !tc, s)
                                   : launch_scores<float>(a, xs, xwide, logits, key, done, !tc, s);
    if (e) return e;
    if ((e = launch_kernel(k_moe_pick, dim3(a.M), kPickThreads, 1, 0, true, s, logits, key, a.M, a.E, a.top, (int)(a.score == KDA_SCORE_SIGMOID),
                           a.scale, ids, weights, done, lists, a.ids, a.weights)))
        return e;
    if (mx) {
        e = launch_experts_tc<true>(a, p, lists, x, xs, xwide, weights, parts, most, columns, s);
    } else if (tc) {
        e = launch_experts_tc<false>(a, p, lists, x, xs, xwide, weights, parts, most, columns, s);
    } else {
        const int sb = a.scale_dtype == KDA_BF16 ? 2 : 4;
        Experts in = {}, out = {};
        in.w = Weights{static_cast<const uint8_t*>(a.w_in), static_cast<const uint8_t*>(a.w_in_scales)};
        in.w_bytes = (int64_t)a.F * a.D, in.s_bytes = (int64_t)2 * a.F * (a.D / a.group) * sb;
        in.x = columns_at(ws + p.x_columns, a.M, a.D);
        in.rows = 2 * a.F, in.K = a.D, in.group = a.group, in.lists = lists, in.E = a.E, in.top = a.top;
        out = in;
        out.w = Weights{static_cast<const uint8_t*>(a.w_out), static_cast<const uint8_t*>(a.w_out_scales)};
        out.w_bytes = (int64_t)a.D * a.F / 2, out.s_bytes = (int64_t)a.D * (a.F / a.group) * sb;
        out.x = columns_at(ws + p.hidden, 2 * (int64_t)slots, a.F);
        out.rows = a.D, out.K = a.F;
        const Direct given{nullptr, nullptr, x, xs, weights};
        // 16 columns where an expert may have more than four tokens (7 tokens of 3 of 33 experts, called one after another: 39 us with 8, 42 with 16)
        e = columns <= 4 ? launch_codes<1>(sb == 2, a.group, a, in, out, given, weights, parts, most, s)
                         : launch_codes<2>(sb == 2, a.group, a, in, out, given, weights, parts, most, s);
    }
    if (e) return e;
    const dim3 grid((a.D + 1023) / 1024, a.M);
    if (a.y_dtype == KDA_BF16) return launch_kernel(k_moe_sum<bf16>, grid, 256, 1, 0, true, s, parts, a.M, a.D, a.top, static_cast<bf16*>(a.y), ys);
    return launch_kernel(k_moe_sum<float>, grid, 256, 1, 0, true, s, parts, a.M, a.D, a.top, static_cast<float*>(a.y), ys);
}

}  // namespace kda
