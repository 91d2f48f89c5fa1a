// kda_verify.cu -- which drafted tokens stand, and the token that follows them.
//
// Rows i of a sequence: draft i is taken while u_i q_i(d_i) < p_i(d_i), compared without rounding the
// product; the first that is not stops the sequence at row a.  The new token is drawn from the residual
//   r = max(p_a - q_a, 0)      (q a single 1 at d_a for a drafter that proposes its best token only)
// or, when every draft stands, from p of the last row, with the last row's u: the first token whose running
// sum is above u times the sum of all.  Without anything left in r, p_a itself is drawn from.
//
// Bound by the one pair of rows per sequence that is read: N V 8 bytes.  The sums decide which token comes out, so
// they are kept in pairs of fp32 (kda_wide.cuh).  Every 1,024 tokens leave one sum in shared memory: the pass over the
// row happens once, and only the run of 1,024 that holds the threshold is read again.  The CTAs of a cluster share a
// row.  256 sequences, 160,000 fp32 tokens: 50 to 52 us (6.3 to 6.5 TB/s); one sequence: 10 us, latency.
#include <cooperative_groups.h>

#include "kda_serve.cuh"
#include "kda_wide.cuh"

namespace kda {

namespace {

namespace cg = cooperative_groups;

constexpr int kTile = 1024;        // tokens per sum
constexpr int kMaxTiles = 4096;    // of one CTA
constexpr int kEnough = 2;         // CTAs per SM that a row is shared for
constexpr int kNotFinite = -2;     // in place of the rank that holds the token, -1 where there is none
constexpr unsigned kAll = 0xffffffffu;

// s += p - q where that is positive (neither is negative).
__device__ __forceinline__ void add_rest(Sum2& s, float p, float q) {
    const float m = fmaxf(p, q), v = m - q;
    s.lo += (m - v) - q;
    s.add(v);
}

template <typename T> struct Pack { static constexpr int width = 16 / sizeof(T); };

// 16 bytes as probabilities; NaN and negative values count as 0.
template <typename T> __device__ __forceinline__ void unpack16(const uint4& r, float (&v)[Pack<T>::width]) {
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        if constexpr (sizeof(T) == 4) {
            v[j] = fmaxf(__uint_as_float(w[j]), 0.f);
        } else {
            v[2 * j] = fmaxf(__uint_as_float(w[j] << 16), 0.f);
            v[2 * j + 1] = fmaxf(__uint_as_float(w[j] & 0xffff0000u), 0.f);
        }
    }
}

// The same of elements i and on, zeros outside the row.
template <typename T> __device__ __forceinline__ void load_edge(const T* row, int64_t i, int V, float (&v)[Pack<T>::width]) {
#pragma unroll
    for (int j = 0; j < Pack<T>::width; ++j) v[j] = i + j >= 0 && i + j < V ? fmaxf(to_f(row[i + j]), 0.f) : 0.f;
}

struct Verify {
    const void* target;
    int64_t target_stride;
    const void* draft;
    int64_t draft_stride;
    const void* tokens;
    const float* u;
    const int32_t* cu;
    int N, V, ranks;
    int64_t T_total;
    void* out;
    int32_t* accepted;
};

// Of a row pair: what is drawn from.  kind 0: p; 1: max(p - q, 0); 2: p without token `hole`.
template <typename T> struct Rest {
    const T *p, *q;
    int kind, hole, V;
    bool wide;
    int shift;  // elements between the row's start and the 16-byte boundary in front of it
    // Adds `Steps` accesses of W tokens, `stride` apart, to a sum.  Where all of [from, to) is inside the row the loads
    // stand in front of the sums, without a branch between them, and are on their way together.
    template <int Steps, int Unroll> __device__ __forceinline__ void sum(Sum2& s, int64_t i, int stride, int64_t from, int64_t to) const {
        constexpr int W = Pack<T>::width;
        if (wide && !(kind == 2 && hole >= from && hole < to) && from >= 0 && to <= V) {
            for (int k0 = 0; k0 < Steps; k0 += Unroll) {
                uint4 pr[Unroll], qr[Unroll];
#pragma unroll
                for (int k = 0; k < Unroll; ++k) pr[k] = __ldg(reinterpret_cast<const uint4*>(p + i + (k0 + k) * stride));
                if (kind == 1) {
#pragma unroll
                    for (int k = 0; k < Unroll; ++k) qr[k] = __ldg(reinterpret_cast<const uint4*>(q + i + (k0 + k) * stride));
                } else {
#pragma unroll
                    for (int k = 0; k < Unroll; ++k) qr[k] = make_uint4(0, 0, 0, 0);
                }
#pragma unroll
                for (int k = 0; k < Unroll; ++k) {
                    float pv[W], qv[W];
                    unpack16<T>(pr[k], pv);
                    unpack16<T>(qr[k], qv);
#pragma unroll
                    for (int j = 0; j < W; ++j) add_rest(s, pv[j], qv[j]);
                }
            }
        } else {
#pragma unroll 4
            for (int k = 0; k < Steps; ++k) {
                float pv[W], qv[W];
                const int64_t at = i + k * stride;
                load_edge(p, at, V, pv);
                if (kind == 1) {
                    load_edge(q, at, V, qv);
                } else {
#pragma unroll
                    for (int j = 0; j < W; ++j) {
                        qv[j] = 0.f;
                        if (kind == 2 && at + j == hole) pv[j] = 0.f;
                    }
                }
#pragma unroll
                for (int j = 0; j < W; ++j) add_rest(s, pv[j], qv[j]);
            }
        }
    }
    __device__ __forceinline__ Wide one(int64_t i) const {  // of one token
        if (i < 0 || i >= V || (kind == 2 && i == hole)) return Wide{};
        Sum2 s;
        add_rest(s, fmaxf(to_f(p[i]), 0.f), kind == 1 ? fmaxf(to_f(q[i]), 0.f) : 0.f);
        return kda::wide(s);
    }
};

// Running sums of the lanes' values, this lane's own included.
__device__ __forceinline__ Wide running(Wide v, int lane) {
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const Wide w{__shfl_up_sync(kAll, v.hi, o), __shfl_up_sync(kAll, v.lo, o)};
        if (lane >= o) v = add(w, v);
    }
    return v;
}

// The sum in front of a lane.
__device__ __forceinline__ Wide in_front(Wide end, int lane) {
    const Wide w{__shfl_up_sync(kAll, end.hi, 1), __shfl_up_sync(kAll, end.lo, 1)};
    return lane ? w : Wide{};
}

// The first lane whose part is above 0 and ends above the threshold; rounding may leave none: then the last lane
// with a part.  -1: no lane has one.
__device__ __forceinline__ int holder(Wide part, Wide end, Wide threshold) {
    const unsigned past = __ballot_sync(kAll, part.hi > 0.f && above(end, threshold)), with = __ballot_sync(kAll, part.hi > 0.f);
    return past ? __ffs(past) - 1 : 31 - __clz(with);
}

// u q < p without rounding the product (the smallest values scaled up, so that its lower half does not vanish).  What is not above 0
// counts as 0 here as in the sums, NaN too.
__device__ __forceinline__ bool takes(float u, float q, float p) {
    q = fmaxf(q, 0.f), p = fmaxf(p, 0.f);
    if (p < 0x1p-60f) p *= 0x1p64f, u *= 0x1p64f;  // u, not q, which may be anything where values need not sum to 1
    const float v = u * q;
    return v < p || (v == p && fmaf(u, q, -v) < 0.f);
}

// Few sequences: 512 threads and a whole tile on its way per warp, for the shortest chain of latencies (one sequence of
// 160,000 tokens: 10.4 us, 10.7 with 256).  Many: 256 threads, three CTAs per SM, so that one's start and search run
// beside the others' reads (256 sequences: 51 us, 77 with 512).
template <typename T, typename Tok, int kThreads> __global__ void __launch_bounds__(kThreads, kThreads == 512 ? 1 : 3) k_verify(const Verify a) {
    constexpr int W = Pack<T>::width, kSteps = kTile / (32 * W), kWarps = kThreads / 32, kUnroll = kThreads == 512 && kSteps == 8 ? 8 : 4;
    __shared__ Wide tile_sum[kMaxTiles];
    __shared__ Wide total_here;
    __shared__ int stop_at, s_owner, found;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int n = blockIdx.x / a.ranks, rank = blockIdx.x % a.ranks;
    const int64_t first = a.cu[n], last = a.cu[n + 1] - 1;
    if (first < 0 || last < first || last >= a.T_total) {  // no rows (or an inconsistent cu_seqlens): the whole cluster
        if (rank == 0 && threadIdx.x == 0) a.accepted[n] = 0;
        return;
    }
    const Tok* tokens = static_cast<const Tok*>(a.tokens);
    const T* target = static_cast<const T*>(a.target);
    const T* draft = static_cast<const T*>(a.draft);
    if (threadIdx.x == 0) stop_at = (int)(last - first);
    __syncthreads();
    for (int64_t i = first + threadIdx.x; i < last; i += kThreads) {
        const int64_t d = (int64_t)tokens[i];
        bool take = false;
        if (d >= 0 && d < a.V) {  // no other token is ever proposed
            const float p = to_f(target[i * a.target_stride + d]);
            take = takes(a.u[i], draft ? to_f(draft[i * a.draft_stride + d]) : 1.f, p);
        }
        if (!take) atomicMin(&stop_at, (int)(i - first));
    }
    __syncthreads();
    const int64_t row = first + stop_at;
    const int64_t d = row < last ? (int64_t)tokens[row] : -1;
    Rest<T> rest;
    rest.p = target + row * a.target_stride;
    rest.q = draft ? draft + row * a.draft_stride : nullptr;
    rest.V = a.V;
    rest.kind = row == last ? 0 : draft ? 1 : 2;
    rest.hole = d >= 0 && d < a.V ? (int)d : -1;
    const uintptr_t mis = reinterpret_cast<uintptr_t>(rest.p) & 15;
    rest.wide = rest.kind != 1 || (reinterpret_cast<uintptr_t>(rest.q) & 15) == mis;
    rest.shift = rest.wide ? (int)(mis / sizeof(T)) : 0;

    const int tiles = (a.V + rest.shift + kTile - 1) / kTile;
    const int t0 = (int)((int64_t)tiles * rank / a.ranks), t1 = (int)((int64_t)tiles * (rank + 1) / a.ranks), own = t1 - t0;
    cg::cluster_group cluster = cg::this_cluster();
    const int per = (own + 31) / 32, l0 = min(lane * per, own), l1 = min(l0 + per, own);  // tiles of a lane of warp 0
    Wide before, threshold, part, end;
    for (;;) {
        for (int t = t0 + warp; t < t1; t += kWarps) {
            Sum2 s;
            const int64_t at = (int64_t)t * kTile - rest.shift;
            rest.template sum<kSteps, kUnroll>(s, at + lane * W, 32 * W, at, at + kTile);
#pragma unroll
            for (int o = 16; o; o >>= 1) {
                const float h = __shfl_xor_sync(kAll, s.hi, o), l = __shfl_xor_sync(kAll, s.lo, o);
                s.add(h);
                s.lo += l;
            }
            if (lane == 0) tile_sum[t - t0] = wide(s);
        }
        __syncthreads();
        if (warp == 0) {
            part = Wide{};
            for (int t = l0; t < l1; ++t) part = add(part, tile_sum[t]);
            end = running(part, lane);
            if (lane == 31) total_here = end;
        }
        if (a.ranks > 1) cluster.sync(); else __syncthreads();
        if (warp == 0) {
            Wide total;
            if (lane < a.ranks) total = a.ranks > 1 ? *cluster.map_shared_rank(&total_here, lane) : total_here;
            const Wide upto = running(total, lane);
            threshold = times(Wide{a.u[last], 0.f}, from(kAll, upto, 31));
            // kNotFinite: an infinity, or a sum beyond fp32, has no share of anything
            const int owner = __shfl_sync(kAll, upto.hi, 31) < INFINITY ? holder(total, upto, threshold) : kNotFinite;
            before = from(kAll, in_front(upto, lane), owner < 0 ? 0 : owner);
            if (lane == 0) s_owner = owner;
        }
        if (a.ranks > 1) cluster.sync(); else __syncthreads();
        if (s_owner != -1 || rest.kind == 0) break;
        rest.kind = 0;  // nothing is left of the residual: p itself
    }
    const int owner = s_owner;
    if (owner < 0 ? rank != 0 : rank != owner) return;
    if (warp == 0) {
        int pick = -1;
        if (owner >= 0) {
            // the lane's tiles, then the tile, then the lane's share of it, then the token
            end = add(before, end);
            int src = holder(part, end, threshold), tile = 0;
            Wide at = in_front(end, lane);
            if (lane == 0) at = before;
            if (lane == src) {
                int left = 0;  // the lane's tiles that hold anything
                for (int t = l0; t < l1; ++t) left += tile_sum[t].hi > 0.f;
                for (int t = l0; t < l1; ++t) {
                    if (!(tile_sum[t].hi > 0.f)) continue;
                    tile = t;
                    const Wide to = add(at, tile_sum[t]);
                    if (above(to, threshold) || --left == 0) break;
                    at = to;
                }
            }
            tile = __shfl_sync(kAll, tile, src);
            at = from(kAll, at, src);
            constexpr int kShare = kTile / 32;
            const int64_t base = (int64_t)(t0 + tile) * kTile - rest.shift;
            Sum2 s;
            rest.template sum<kShare / W, 4>(s, base + lane * kShare, W, base, base + kTile);
            part = wide(s);
            end = add(at, running(part, lane));
            src = holder(part, end, threshold);
            const Wide front = in_front(end, lane);
            at = from(kAll, lane ? front : at, src);
            const int64_t token = base + src * kShare + lane;  // kShare is 32
            part = rest.one(token);
            end = add(at, running(part, lane));
            src = holder(part, end, threshold);
            pick = (int)__shfl_sync(kAll, token, src);
        }
        if (lane == 0) found = pick;
    }
    __syncthreads();
    Tok* out = static_cast<Tok*>(a.out);
    for (int64_t i = first + threadIdx.x; i <= last; i += kThreads) out[i] = i < row ? tokens[i] : i == row ? (Tok)found : (Tok)-1;
    if (threadIdx.x == 0) a.accepted[n] = stop_at;
}

template <typename T, typename Tok, int kThreads> cudaError_t launch_threads(const kda_verify_args& a, int ranks, cudaStream_t s) {
    Verify p;
    p.target = a.target, p.target_stride = a.target_stride ? a.target_stride : a.V;
    p.draft = a.draft, p.draft_stride = a.draft_stride ? a.draft_stride : a.V;
    p.tokens = a.tokens, p.u = a.u, p.cu = a.cu_seqlens;
    p.N = a.N, p.V = a.V, p.T_total = a.T_total, p.out = a.out, p.accepted = a.accepted;
    p.ranks = ranks;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = ranks;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(a.N * ranks));
    cfg.blockDim = kThreads;
    cfg.stream = s;
    cfg.attrs = at;
    cfg.numAttrs = ranks > 1 ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, k_verify<T, Tok, kThreads>, p);
}

template <typename T, typename Tok> cudaError_t launch(const kda_verify_args& a, cudaStream_t s) {
    int ranks = 1;
    while (ranks < 8 && (int64_t)a.N * ranks < kEnough * 152 && a.V / kTile >= 2 * ranks) ranks *= 2;
    return (int64_t)a.N * ranks <= 152 ? launch_threads<T, Tok, 512>(a, ranks, s) : launch_threads<T, Tok, 256>(a, ranks, s);
}

}  // namespace

cudaError_t launch_verify(const kda_verify_args& a, cudaStream_t s) {
    if (a.dtype == KDA_BF16) return a.token_bytes == 8 ? launch<bf16, long long>(a, s) : launch<bf16, int>(a, s);
    return a.token_bytes == 8 ? launch<float, long long>(a, s) : launch<float, int>(a, s);
}

}  // namespace kda
