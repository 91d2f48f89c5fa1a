// kda_verify.cu -- which drafted tokens stand, and the token that follows them.
//
// Rows i of a sequence: draft i is taken while u_i q_i(d_i) < p_i(d_i), as products of fp32 in fp64, which
// are exact; the first that is not stops the sequence at row a.  The new token is drawn from the residual
//   r = max(p_a - q_a, 0)      (q a single 1 at d_a for a drafter that proposes its best token only)
// or, when every draft stands, from p of the last row, with the last row's u: the first token whose running
// sum is above u times the sum of all.  Without anything left in r, p_a itself is drawn from.
//
// Bound by the one pair of rows per sequence that is read: N V 8 bytes.  The sums decide which token comes out, so
// they are kept in two fp32 (value and rounding; fp64 at its rate here would take longer than the read), and
// every 2,048 tokens leave one sum in shared memory: the pass over the row happens once, and only the
// block of 2,048 that holds the threshold is read again, token by token, in fp64.  The CTAs of a cluster
// share a row where there are few sequences.
#include <cooperative_groups.h>

#include "kda_serve.cuh"

namespace kda {

namespace {

namespace cg = cooperative_groups;

constexpr int kThreads = 512, kWarps = 16;
constexpr int kTile = 2048;        // tokens per sum
constexpr int kMaxTiles = 2048;    // of one CTA

struct Sum2 {  // fp32 value and what its roundings lost
    float hi = 0.f, lo = 0.f;
    __device__ __forceinline__ void add(float v) {
        const float s = hi + v, b = s - hi;
        lo += (hi - (s - b)) + (v - b);
        hi = s;
    }
    __device__ __forceinline__ double value() const { return isfinite(hi) ? (double)hi + (double)lo : (double)hi; }
};

template <typename T> struct Pack { static constexpr int width = 16 / sizeof(T); };

// `width` probabilities from element i of a row (i - first element of an aligned 16 bytes when wide), zeros
// outside the row; NaN and negative values count as 0.
template <typename T> __device__ __forceinline__ void load_row(const T* row, int64_t i, int V, bool wide, float (&v)[Pack<T>::width]) {
    constexpr int W = Pack<T>::width;
    if (wide && i >= 0 && i + W <= V) {
        const uint4 q = __ldg(reinterpret_cast<const uint4*>(row + i));
        if constexpr (sizeof(T) == 4) {
            v[0] = __uint_as_float(q.x), v[1] = __uint_as_float(q.y), v[2] = __uint_as_float(q.z), v[3] = __uint_as_float(q.w);
        } else {
            const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
            for (int j = 0; j < 4; ++j) v[2 * j] = __uint_as_float(w[j] << 16), v[2 * j + 1] = __uint_as_float(w[j] & 0xffff0000u);
        }
    } else {
#pragma unroll
        for (int j = 0; j < W; ++j) v[j] = i + j >= 0 && i + j < V ? to_f(row[i + j]) : 0.f;
    }
#pragma unroll
    for (int j = 0; j < W; ++j) v[j] = v[j] > 0.f ? v[j] : 0.f;
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
    __device__ __forceinline__ void at(int64_t i, float (&v)[Pack<T>::width], float (&q_)[Pack<T>::width]) const {
        load_row(p, i, V, wide, v);
        if (kind == 1) {
            load_row(q, i, V, wide, q_);
        } else {
#pragma unroll
            for (int j = 0; j < Pack<T>::width; ++j) {
                q_[j] = 0.f;
                if (kind == 2 && i + j == hole) v[j] = 0.f;
            }
        }
    }
};

template <typename T, typename Tok> __global__ void __launch_bounds__(kThreads, 2) k_verify(const Verify a) {
    constexpr int W = Pack<T>::width, kSteps = kTile / (32 * W);
    __shared__ double tile_sum[kMaxTiles];
    __shared__ double total_here, before_tile;
    __shared__ int stop_at, found_tile, found;
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
            const double p = (double)to_f(target[i * a.target_stride + d]);
            const double q = draft ? (double)to_f(draft[i * a.draft_stride + d]) : 1.0;
            take = (double)a.u[i] * q < p;
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
    const int t0 = (int)((int64_t)tiles * rank / a.ranks), t1 = (int)((int64_t)tiles * (rank + 1) / a.ranks);
    cg::cluster_group cluster = cg::this_cluster();
    double before = 0.0, threshold = 0.0;
    int owner = -1;
    for (;;) {
        for (int t = t0 + warp; t < t1; t += kWarps) {
            Sum2 s;
#pragma unroll 4
            for (int k = 0; k < kSteps; ++k) {
                float p[W], q[W];
                rest.at((int64_t)t * kTile + (k * 32 + lane) * W - rest.shift, p, q);
#pragma unroll
                for (int j = 0; j < W; ++j) {
                    const float v = p[j] - q[j];
                    if (v > 0.f) {
                        s.lo += (p[j] - v) - q[j];
                        s.add(v);
                    }
                }
            }
#pragma unroll
            for (int o = 16; o; o >>= 1) {
                const float h = __shfl_xor_sync(0xffffffffu, s.hi, o), l = __shfl_xor_sync(0xffffffffu, s.lo, o);
                s.add(h);
                s.lo += l;
            }
            if (lane == 0) tile_sum[t - t0] = s.value();
        }
        __syncthreads();
        if (warp == 0) {
            double s = 0.0;
            for (int t = lane; t < t1 - t0; t += 32) s += tile_sum[t];
#pragma unroll
            for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
            if (lane == 0) total_here = s;
        }
        if (a.ranks > 1) cluster.sync(); else __syncthreads();
        double total = 0.0, sums[8];
        for (int r = 0; r < a.ranks; ++r) {
            sums[r] = a.ranks > 1 ? *cluster.map_shared_rank(&total_here, r) : total_here;
            total += sums[r];
        }
        threshold = (double)a.u[last] * total;
        before = 0.0;
        owner = -1;
        int last_with = -1;
        double run = 0.0;
        for (int r = 0; r < a.ranks; ++r) {
            if (sums[r] > 0.0) {
                last_with = r;
                if (owner < 0 && run + sums[r] > threshold) owner = r, before = run;
            }
            run += sums[r];
        }
        if (owner < 0 && last_with >= 0) {  // rounding, or a sum that is not finite: the last part that holds anything
            owner = last_with;
            before = threshold;
        }
        if (a.ranks > 1) cluster.sync(); else __syncthreads();
        if (owner >= 0 || rest.kind == 0) break;
        rest.kind = 0;  // nothing is left of the residual: p itself
    }
    if (owner < 0 ? rank == 0 : rank == owner) {
        if (threadIdx.x == 0) {
            found = -1;
            found_tile = -1;
            double run = before;
            int last_with = -1;
            for (int t = 0; t < t1 - t0 && owner >= 0; ++t) {
                if (!(tile_sum[t] > 0.0)) continue;
                last_with = t;
                if (run + tile_sum[t] > threshold) {
                    found_tile = t;
                    before_tile = run;
                    break;
                }
                run += tile_sum[t];
            }
            if (found_tile < 0 && last_with >= 0) {
                found_tile = last_with;
                before_tile = run - tile_sum[last_with];
            }
        }
        __syncthreads();
        if (warp == 0 && found_tile >= 0) {
            // a lane takes kTile / 32 tokens in a row; the first lane whose running sum passes the threshold holds the token
            const int64_t base = (int64_t)(t0 + found_tile) * kTile + lane * (kTile / 32) - rest.shift;
            double s = 0.0;
            for (int k = 0; k < kTile / 32 / W; ++k) {
                float p[W], q[W];
                rest.at(base + k * W, p, q);
#pragma unroll
                for (int j = 0; j < W; ++j)
                    if (p[j] > q[j]) s += (double)p[j] - (double)q[j];
            }
            double run = s;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const double v = __shfl_up_sync(0xffffffffu, run, o);
                if (lane >= o) run += v;
            }
            const double upto = before_tile + (run - s);
            const unsigned over = __ballot_sync(0xffffffffu, s > 0.0 && before_tile + run > threshold);
            const unsigned with = __ballot_sync(0xffffffffu, s > 0.0);
            const int holder = over ? __ffs(over) - 1 : 31 - __clz(with | 1u);
            if (lane == holder) {
                double sum = upto;
                int pick = -1;
                bool done = false;
                for (int k = 0; k < kTile / 32 / W && !done; ++k) {
                    float p[W], q[W];
                    rest.at(base + k * W, p, q);
#pragma unroll
                    for (int j = 0; j < W; ++j) {
                        if (done || !(p[j] > q[j])) continue;
                        sum += (double)p[j] - (double)q[j];
                        pick = (int)(base + k * W + j);  // the last one with a share, should rounding leave the threshold above all
                        done = sum > threshold;
                    }
                }
                found = pick;
            }
        }
        __syncthreads();
        Tok* out = static_cast<Tok*>(a.out);
        for (int64_t i = first + threadIdx.x; i <= last; i += kThreads) out[i] = i < row ? tokens[i] : i == row ? (Tok)found : (Tok)-1;
        if (threadIdx.x == 0) a.accepted[n] = stop_at;
    }
}

template <typename T, typename Tok> cudaError_t launch(const kda_verify_args& a, cudaStream_t s) {
    Verify p;
    p.target = a.target, p.target_stride = a.target_stride ? a.target_stride : a.V;
    p.draft = a.draft, p.draft_stride = a.draft_stride ? a.draft_stride : a.V;
    p.tokens = a.tokens, p.u = a.u, p.cu = a.cu_seqlens;
    p.N = a.N, p.V = a.V, p.T_total = a.T_total, p.out = a.out, p.accepted = a.accepted;
    // CTAs for about two per SM, and at least a tile per warp
    int ranks = 1;
    while (ranks < 8 && (int64_t)a.N * ranks < 2 * 152 && a.V / kTile >= 2 * ranks * kWarps / 4) ranks *= 2;
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
    return cudaLaunchKernelEx(&cfg, k_verify<T, Tok>, p);
}

}  // namespace

cudaError_t launch_verify(const kda_verify_args& a, cudaStream_t s) {
    if (a.dtype == KDA_BF16) return a.token_bytes == 8 ? launch<bf16, long long>(a, s) : launch<bf16, int>(a, s);
    return a.token_bytes == 8 ? launch<float, long long>(a, s) : launch<float, int>(a, s);
}

}  // namespace kda
