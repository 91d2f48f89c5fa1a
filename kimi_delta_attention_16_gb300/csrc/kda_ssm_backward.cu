// kda_ssm_backward.cu -- the gradients of the selective state space scan.
//
//   g_t = dy_t silu(z_t);  lambda_t = C_t g_t + a_{t+1} lambda_{t+1};  q_t = a_{t+1} lambda_{t+1}
//   dC_t = sum_c g h_t;  dB_t = sum_c lambda delta u;  dA += lambda a h_{t-1} delta
//   s1 = sum_n lambda B;  s2 = sum_n lambda a h_{t-1} A
//   du = delta s1 + D g;  ddelta = u s1 + s2;  dz = dy (sum_n C h + D u) silu'(z)
//
// The states are recomputed.  Forward passes leave the state in front of every fourth token; the
// main kernel walks a piece of the token axis backwards in tiles of four, runs a tile forward from
// its checkpoint with the state in front of each token in registers (so that q_t h_{t-1} needs no decayed
// state), and then backward.  Where a stream is cut into pieces, what enters a piece from the right
// comes from a pass of its own (k_rev), the mirror image of the forward scan's
// (4,096 tokens in sequences of 128: 68 -> 38 us, since a piece's first border ends it).
//
// Two sums cross the threads for every token: over the states (s1, s2, y of a channel) and over the
// channels (dB, dC of a state).  A thread therefore holds a 4 x 4 tile of (channel, state): both
// sums run over four values in registers first, which costs nothing (they ride on the products),
// and the rest goes through shared memory.  Sums over the blocks' channels and over the pieces go
// through the workspace and are added in a fixed order.
//
// Measured, 4,096 x 4,096 x 16 bf16 with the gate: 543 us = pieces' own states 55, checkpoints 72,
// k_rev 69, the main kernel 320, joins and sums 27.  The main kernel issues an instruction in 40 %
// of the cycles: two blocks of 255-register threads per SM (112 bytes spilled with 16 states, 44 with 8, 16 with 32)
// leave two warps per scheduler, whose dependent instructions wait for one another.  Three blocks (168 registers) spill: 640 us; 2 channels x 4 states
// per thread (four blocks of 128 registers) 356, its cross-thread sums cost what the warps gain.
// In a copy without them: the border path 18 us, dB and dC across threads 42, the elementwise end
// of a tile 68, the copies 60.
#include "kda_ssm.cuh"

namespace kda {

namespace {

using namespace ssm;

struct BParams {
    Params f;
    const void* dy;
    int64_t dys;
    const float* dfin;
    float *rev, *rsum, *pa, *pd, *pbc, *dinit;
    void *du, *ddt, *dz;
    int bpg;  // blocks per group of the main kernel
    bool vec;   // 16-byte copies of every row, dy's too
    bool wide;  // two channels per access to du, ddt and dz
};

// ------------------------------------------------------------------ what enters a piece from the right
// Pieces 1 .. pieces - 1, each from zero at its right end (or from d_final_state where a sequence
// ends; what lies behind the first end is passed over): q in front of its first token, and its sum of delta.  Layout and copies as in the forward scan.
template <typename T, int NS>
__global__ void __launch_bounds__(Lay<NS, 1>::NT, 8) k_rev(BParams b) {
    using Y = Lay<NS, 1>;
    constexpr int TT = Y::TT, NT = Y::NT, BPT = Y::BPT, H = Y::SPT / 2, Q = Y::SPT / 4, CB = Y::CB;
    constexpr int kDepth = 4;
    struct Tile {
        T dt[TT][CB], dy[TT][CB], z[TT][CB], C[TT][NS];
    };
    __shared__ __align__(16) Tile ring[kDepth];
    __shared__ __align__(16) float sC[2][TT][NS];
    const Params& p = b.f;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int l = lane / Y::KPW, cl = warp * Y::KPW + lane % Y::KPW;
    const int bpg = (p.Cg + CB - 1) / CB, g = blockIdx.x / bpg;  // blocks per group
    const int c_lo = g * p.Cg + (blockIdx.x % bpg) * CB, c_hi = (g + 1) * p.Cg, cols = c_hi - c_lo;
    const bool in = c_lo + cl < c_hi, gate = p.z != nullptr;
    const int c = in ? c_lo + cl : c_hi - 1;
    const int piece = blockIdx.y + 1;
    const int64_t t0 = piece * p.piece;
    int64_t t1 = t0 + p.piece < p.T ? t0 + p.piece : p.T;
    const int64_t so = (int64_t)c * NS + l * Y::SPT;
    f2 A2[H], q[H];
#pragma unroll
    for (int i = 0; i < Q; ++i) {
        const float4 a = __ldg(reinterpret_cast<const float4*>(p.A + so) + i);
        A2[2 * i] = f2_of(a.x * kLog2e, a.y * kLog2e);
        A2[2 * i + 1] = f2_of(a.z * kLog2e, a.w * kLog2e);
    }
    auto load_q = [&](const float* base, int64_t n) {
#pragma unroll
        for (int i = 0; i < Q; ++i) {
            float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
            if (base) s = reinterpret_cast<const float4*>(base + n * p.C * NS + so)[i];
            q[2 * i] = f2_of(s.x, s.y);
            q[2 * i + 1] = f2_of(s.z, s.w);
        }
    };
    const float bias = p.dt_bias ? p.dt_bias[c] : 0.f;
    int tiles = (int)((t1 - t0 + TT - 1) / TT);
    auto issue = [&](int j) {  // the j-th tile from the right
        if (j < tiles) {
            Tile& r = ring[j % kDepth];
            const int64_t tb = t0 + (int64_t)(tiles - 1 - j) * TT;
            const int rows = (int)(t1 - tb < TT ? t1 - tb : TT);
            const uint32_t row = (uint32_t)tb;
            copy_tile<T, TT, CB, NT>(&r.dt[0][0], static_cast<const T*>(p.dt) + c_lo, p.dts, row, rows, cols, b.vec);
            copy_tile<T, TT, CB, NT>(&r.dy[0][0], static_cast<const T*>(b.dy) + c_lo, b.dys, row, rows, cols, b.vec);
            if (gate)
                copy_tile<T, TT, CB, NT>(&r.z[0][0], static_cast<const T*>(p.z) + c_lo, p.zs, row, rows, cols, b.vec);
            copy_tile<T, TT, NS, NT>(&r.C[0][0], static_cast<const T*>(p.Cm) + g * NS, p.cs, row, rows, NS, b.vec);
        }
        cp_commit();
    };
    auto widen = [&](int j) {
        const Tile& r = ring[j % kDepth];
#pragma unroll
        for (int k = 0; k < BPT; ++k) {
            const int i = k * NT + tid;
            sC[j & 1][i / NS][i % NS] = to_f(r.C[i / NS][i % NS]);
        }
    };
#pragma unroll
    for (int j = 0; j < kDepth - 1; ++j) issue(j);
    if (p.N > 1) {  // the sequence that comes in from the left is all that sends a gradient there: from its end on
        const int64_t e = p.cu[seq_of(p.cu, p.N, t0) + 1];
        if (e <= t1 - TT && e > t0) {
            tiles = (int)((e - t0 + TT - 1) / TT);
            if (t0 + (int64_t)tiles * TT < t1) t1 = t0 + (int64_t)tiles * TT;
            cp_wait<0>();  // those copies are not wanted
            __syncthreads();
#pragma unroll
            for (int j = 0; j < kDepth - 1; ++j) issue(j);
        }
    }
    int n = seq_of(p.cu, p.N, t1 - 1);
    int64_t s0 = p.cu[n];
    load_q(p.cu[n + 1] == t1 ? b.dfin : nullptr, n);
    cp_wait<kDepth - 2>();
    __syncthreads();
    widen(0);
    float dsum = 0.f;
    for (int j = 0; j < tiles; ++j) {
        const int64_t tb = t0 + (int64_t)(tiles - 1 - j) * TT;
        const int buf = j & 1;
        cp_wait<kDepth - 3>();
        __syncthreads();
        if (j + 1 < tiles) widen(j + 1);
        issue(j + kDepth - 1);
        const Tile& r = ring[j % kDepth];
        const int nt = (int)(t1 - tb < TT ? t1 - tb : TT);
        auto token = [&](int t, float d, float gv) {
            const f2 dd = f2_dup(d), gg = f2_dup(gv);
#pragma unroll
            for (int i = 0; i < Q; ++i) {
                const float4 v = *reinterpret_cast<const float4*>(&sC[buf][t][l * Y::SPT + 4 * i]);
                q[2 * i] = mul2(exp2_2(mul2(dd, A2[2 * i])), fma2(f2_of(v.x, v.y), gg, q[2 * i]));
                q[2 * i + 1] = mul2(exp2_2(mul2(dd, A2[2 * i + 1])), fma2(f2_of(v.z, v.w), gg, q[2 * i + 1]));
            }
        };
        auto grad = [&](int t) {
            const float d = to_f(r.dy[t][cl]);
            return gate ? d * silu(to_f(r.z[t][cl])) : d;
        };
        if (nt == TT && s0 <= tb) {  // no sequence starts behind the tile's first token
            float d[TT], gv[TT];
#pragma unroll
            for (int t = 0; t < TT; t += 2) {
                const f2 x = add2(f2_of(to_f(r.dt[t][cl]), to_f(r.dt[t + 1][cl])), f2_dup(bias));
                const f2 v = p.softplus ? softplus2(x) : x;
                d[t] = f2_lo(v);
                d[t + 1] = f2_hi(v);
                gv[t] = grad(t);
                gv[t + 1] = grad(t + 1);
            }
#pragma unroll
            for (int t = TT - 1; t >= 0; --t) {
                token(t, d[t], gv[t]);
                dsum += d[t];
            }
        } else {
#pragma unroll 1
            for (int t = nt - 1; t >= 0; --t) {
                if (tb + t < s0) {  // into the sequence before
                    n = seq_of(p.cu, p.N, tb + t);
                    s0 = p.cu[n];
                    load_q(b.dfin, n);
                }
                const float x = to_f(r.dt[t][cl]) + bias, d = p.softplus ? softplus(x) : x;
                token(t, d, grad(t));
                dsum += d;
            }
        }
    }
    if (in) {
#pragma unroll
        for (int i = 0; i < Q; ++i)
            reinterpret_cast<float4*>(b.rev + (int64_t)piece * p.C * NS + so)[i] =
                make_float4(f2_lo(q[2 * i]), f2_hi(q[2 * i]), f2_lo(q[2 * i + 1]), f2_hi(q[2 * i + 1]));
        if (l == 0) b.rsum[(int64_t)piece * p.C + c] = dsum;
    }
}

// Slot k: from what piece k sends to its left by itself to all that it sends (what piece k - 1 starts from).
template <int NS> __global__ void __launch_bounds__(kJoinThreads) k_rev_join(BParams b) {
    const Params& p = b.f;
    __shared__ uint32_t closed[kJoinBits / 32];
    mark_closed<-1>(p, closed);
    const int64_t i = (int64_t)blockIdx.x * kJoinThreads + threadIdx.x, row = (int64_t)p.C * NS;
    if (i >= row) return;
    const float a2 = p.A[i] * kLog2e;
    float* slot = b.rev + i;
    const float* sum = b.rsum + i / NS;
    join<-1>(p, closed, p.pieces - 2, p.pieces - 2, a2, slot[(p.pieces - 1) * row], slot, sum, row);
}

// ------------------------------------------------------------------ the main kernel
// Block of CH channels x NS states, 4 x 4 per thread; lanes with the same states are neighbours.
template <int NS> struct BLay {
    static constexpr int L = NS / 4;            // threads along the states
    static constexpr int NT = 128;
    static constexpr int KK = NT / L;           // threads along the channels
    static constexpr int KPW = 32 / L;
    static constexpr int CH = 4 * KK;           // channels per block
    static constexpr int TT = 4;                // tokens per tile
    // Elementwise work: a thread has the same two channels of every RPT-th token of the tile.
    static constexpr int PR = CH / 2, RPT = NT / PR, PPT = RPT < TT ? TT / RPT : 1;
    static constexpr int RPC = RPT < TT ? RPT : TT;  // threads that share a channel (NS = 64: half of them idle)
    static constexpr int BPT = (TT * NS + NT - 1) / NT;
    static constexpr int VW = 2 * NS + 4;       // row of the dB | dC parts, padded against bank conflicts
};
template <typename T, int NS> struct BShared {
    using Y = BLay<NS>;
    struct Tile {
        T u[Y::TT][Y::CH], dt[Y::TT][Y::CH], z[Y::TT][Y::CH], dy[Y::TT][Y::CH], B[Y::TT][NS], C[Y::TT][NS];
    };
    Tile ring[2];
    float4 ck[2][4][Y::NT];                       // checkpoints, each thread its own
    float d[Y::TT][Y::CH], du[Y::TT][Y::CH], g[Y::TT][Y::CH];
    float B[Y::TT][NS], C[Y::TT][NS];
    float part[3][Y::TT][Y::L][Y::CH];            // s1, s2, y
    float bc[Y::TT][Y::KK][Y::VW];                // dB | dC
};

template <typename T, int NS>
__global__ void __launch_bounds__(128, 2) k_ssm_bwd(BParams b) {
    using Y = BLay<NS>;
    constexpr int L = Y::L, NT = Y::NT, CH = Y::CH, TT = Y::TT, PPT = Y::PPT;
    extern __shared__ __align__(16) unsigned char raw_shared[];
    BShared<T, NS>& sm = *reinterpret_cast<BShared<T, NS>*>(raw_shared);
    const Params& p = b.f;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int l = lane / Y::KPW, kk = warp * Y::KPW + lane % Y::KPW;
    const int g = blockIdx.x / b.bpg;
    const int c_lo = g * p.Cg + (blockIdx.x % b.bpg) * CH, c_hi = (g + 1) * p.Cg, cols = c_hi - c_lo;
    const int piece = blockIdx.y;
    const int64_t t0 = piece * p.piece, t1 = t0 + p.piece < p.T ? t0 + p.piece : p.T;
    const bool gate = p.z != nullptr;
    const int cc = 2 * (tid % Y::PR), row = tid / Y::PR, c0 = c_lo + cc;  // this thread's two channels, its first token
    const bool in0 = c0 < c_hi, in1 = c0 + 1 < c_hi;
    auto store = [&](void* base, int64_t o, f2 v) {  // this thread's two channels of a row
        T* q = static_cast<T*>(base) + o;
        if (b.wide) {
            put2(q, v);
        } else {
            q[0] = from_f<T>(f2_lo(v));
            if (in1) q[1] = from_f<T>(f2_hi(v));
        }
    };

    // 4 channels x 4 states: pairs run over the channels (0, 1) and (2, 3)
    auto load_tile = [&](const float* base, int64_t row, f2 (&v)[4][2], float scale) {
        float m[4][4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int ch = c_lo + 4 * kk + i;
            float4 f = make_float4(0.f, 0.f, 0.f, 0.f);
            if (base && ch < c_hi) f = *reinterpret_cast<const float4*>(base + (row * p.C + ch) * NS + 4 * l);
            m[i][0] = f.x; m[i][1] = f.y; m[i][2] = f.z; m[i][3] = f.w;
        }
#pragma unroll
        for (int s = 0; s < 4; ++s)
#pragma unroll
            for (int h = 0; h < 2; ++h) v[s][h] = f2_of(m[2 * h][s] * scale, m[2 * h + 1][s] * scale);
    };
    auto store_tile = [&](float* base, int64_t row, const f2 (&v)[4][2]) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int ch = c_lo + 4 * kk + i, h = i / 2;
            float o[4];
#pragma unroll
            for (int s = 0; s < 4; ++s) o[s] = i & 1 ? f2_hi(v[s][h]) : f2_lo(v[s][h]);
            if (ch < c_hi)
                *reinterpret_cast<float4*>(base + (row * p.C + ch) * NS + 4 * l) = make_float4(o[0], o[1], o[2], o[3]);
        }
    };
    f2 A2[4][2], q[4][2], dA[4][2];
    load_tile(p.A, 0, A2, kLog2e);
#pragma unroll
    for (int s = 0; s < 4; ++s) dA[s][0] = dA[s][1] = f2_dup(0.f);
    auto both = [&](const float* v) { return f2_of(v && in0 ? v[c0] : 0.f, v && in1 ? v[c0 + 1] : 0.f); };
    const f2 bias = both(p.dt_bias), skip = both(p.D);
    f2 accD = f2_dup(0.f), accB = accD;
    const int tiles = (int)((t1 - t0 + TT - 1) / TT);
    auto issue = [&](int j) {  // the j-th tile from the right
        if (j < tiles) {
            typename BShared<T, NS>::Tile& r = sm.ring[j & 1];
            const int64_t tb = t0 + (int64_t)(tiles - 1 - j) * TT;
            const int rows = (int)(t1 - tb < TT ? t1 - tb : TT);
            const uint32_t row = (uint32_t)tb;
            copy_tile<T, TT, CH, NT>(&r.u[0][0], static_cast<const T*>(p.u) + c_lo, p.us, row, rows, cols, b.vec);
            copy_tile<T, TT, CH, NT>(&r.dt[0][0], static_cast<const T*>(p.dt) + c_lo, p.dts, row, rows, cols, b.vec);
            copy_tile<T, TT, CH, NT>(&r.dy[0][0], static_cast<const T*>(b.dy) + c_lo, b.dys, row, rows, cols, b.vec);
            if (gate)
                copy_tile<T, TT, CH, NT>(&r.z[0][0], static_cast<const T*>(p.z) + c_lo, p.zs, row, rows, cols, b.vec);
            copy_tile<T, TT, NS, NT>(&r.B[0][0], static_cast<const T*>(p.B) + g * NS, p.bs, row, rows, NS, b.vec);
            copy_tile<T, TT, NS, NT>(&r.C[0][0], static_cast<const T*>(p.Cm) + g * NS, p.cs, row, rows, NS, b.vec);
            const float* ck = p.ckpt + (int64_t)(row / 4) * (uint32_t)(p.C * NS) + (c_lo + 4 * kk) * NS + 4 * l;
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (c_lo + 4 * kk + i < c_hi) cp_async16(&sm.ck[j & 1][i][tid], ck + i * NS);
                else sm.ck[j & 1][i][tid] = make_float4(0.f, 0.f, 0.f, 0.f);  // past the group's last channel
        }
        cp_commit();
    };
    issue(0);
    int n = seq_of(p.cu, p.N, t1 - 1);
    int64_t s0 = p.cu[n];  // start of the sequence that the walk is in
    if (p.cu[n + 1] == t1) load_tile(b.dfin, n, q, 1.f);
    else load_tile(piece + 1 < p.pieces ? b.rev : nullptr, piece + 1, q, 1.f);
    cp_wait<0>();
    __syncthreads();
    for (int j = 0; j < tiles; ++j) {
        const int64_t tb = t0 + (int64_t)(tiles - 1 - j) * TT;
        const int nt = (int)(t1 - tb < TT ? t1 - tb : TT);
        const typename BShared<T, NS>::Tile& r = sm.ring[j & 1];
        // Step sizes and gradients of the reads; tokens past the end and channels past the group count as
        // zeros everywhere, which leaves states, gradients and sums as they are.
#pragma unroll
        for (int i = 0; i < PPT; ++i) {
            const int t = i * Y::RPT + row;
            if (Y::RPT > TT && t >= TT) break;
            const bool on0 = t < nt && in0, on1 = t < nt && in1;
            auto get = [&](const T* v) {
                const f2 w = pair_of(v);
                return f2_of(on0 ? f2_lo(w) : 0.f, on1 ? f2_hi(w) : 0.f);
            };
            const f2 x = add2(get(&r.dt[t][cc]), bias);
            f2 d = p.softplus ? softplus2(x) : x, gv = get(&r.dy[t][cc]);
            d = f2_of(on0 ? f2_lo(d) : 0.f, on1 ? f2_hi(d) : 0.f);
            if (gate) {
                const f2 z = get(&r.z[t][cc]);
                gv = mul2(gv, mul2(z, sigmoid2(z)));
            }
            put2(&sm.d[t][cc], d);
            put2(&sm.du[t][cc], mul2(d, get(&r.u[t][cc])));
            put2(&sm.g[t][cc], gv);
        }
#pragma unroll
        for (int k = 0; k < Y::BPT; ++k) {
            const int i = k * NT + tid;
            if ((TT * NS) % NT && i >= TT * NS) break;
            const bool on = i / NS < nt;
            sm.B[i / NS][i % NS] = on ? to_f(r.B[i / NS][i % NS]) : 0.f;
            sm.C[i / NS][i % NS] = on ? to_f(r.C[i / NS][i % NS]) : 0.f;
        }
        __syncthreads();
        issue(j + 1);

        // The state in front of each token: the tile's first stays in shared memory, the others in registers.
        f2 hs[TT - 1][4][2];
        auto before = [&](int t, f2 (&h)[4][2]) {
#pragma unroll
            for (int s = 0; s < 4; ++s)
#pragma unroll
                for (int k = 0; k < 2; ++k)
                    h[s][k] = t ? hs[t - 1][s][k]
                                : f2_of((&sm.ck[j & 1][2 * k][tid].x)[s], (&sm.ck[j & 1][2 * k + 1][tid].x)[s]);
        };
        auto pair4 = [&](const float* v, f2 (&o)[2]) {  // four channels of a row
            const float4 f = *reinterpret_cast<const float4*>(v + 4 * kk);
            o[0] = f2_of(f.x, f.y);
            o[1] = f2_of(f.z, f.w);
        };
        auto dup4 = [&](const float* v, f2 (&o)[4]) {  // four states of a row, each for both channels of a pair
            const float4 f = *reinterpret_cast<const float4*>(v + 4 * l);
            o[0] = f2_dup(f.x); o[1] = f2_dup(f.y); o[2] = f2_dup(f.z); o[3] = f2_dup(f.w);
        };
        auto forward = [&](int t) {  // the state behind token t
            f2 d[2], du[2], B[4], h[4][2];
            pair4(sm.d[t], d);
            pair4(sm.du[t], du);
            dup4(sm.B[t], B);
            before(t, h);
#pragma unroll
            for (int s = 0; s < 4; ++s)
#pragma unroll
                for (int k = 0; k < 2; ++k)
                    hs[t][s][k] = fma2(du[k], B[s], mul2(exp2_2(mul2(d[k], A2[s][k])), h[s][k]));
        };
        // kKept: the state behind token t is what stands in front of the next one.
        auto backward = [&](int t, auto kept) {
            f2 d[2], du[2], gg[2], B[4], C[4], s1[2], s2[2], y[2], h[4][2];
            before(t, h);
            pair4(sm.d[t], d);
            pair4(sm.du[t], du);
            pair4(sm.g[t], gg);
            dup4(sm.B[t], B);
            dup4(sm.C[t], C);
            float dB[4], dC[4];
#pragma unroll
            for (int k = 0; k < 2; ++k) s1[k] = s2[k] = y[k] = f2_dup(0.f);
#pragma unroll
            for (int s = 0; s < 4; ++s) {
                f2 vb = f2_dup(0.f), vc = f2_dup(0.f);
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const f2 a = exp2_2(mul2(d[k], A2[s][k])), lam = fma2(C[s], gg[k], q[s][k]);
                    f2 hk;
                    if constexpr (kept) hk = hs[t < TT - 1 ? t : 0][s][k];
                    else hk = fma2(du[k], B[s], mul2(a, h[s][k]));
                    q[s][k] = mul2(a, lam);
                    vc = fma2(gg[k], hk, vc);
                    vb = fma2(lam, du[k], vb);
                    y[k] = fma2(C[s], hk, y[k]);
                    s1[k] = fma2(lam, B[s], s1[k]);
                    const f2 w = mul2(q[s][k], h[s][k]);
                    s2[k] = fma2(w, A2[s][k], s2[k]);
                    dA[s][k] = fma2(w, d[k], dA[s][k]);
                }
                dB[s] = f2_lo(vb) + f2_hi(vb);
                dC[s] = f2_lo(vc) + f2_hi(vc);
            }
            auto put = [&](float* row, const f2 (&v)[2]) {
                *reinterpret_cast<float4*>(row + 4 * kk) = make_float4(f2_lo(v[0]), f2_hi(v[0]), f2_lo(v[1]), f2_hi(v[1]));
            };
            put(sm.part[0][t][l], s1);
            put(sm.part[1][t][l], s2);
            put(sm.part[2][t][l], y);
            *reinterpret_cast<float4*>(&sm.bc[t][kk][4 * l]) = make_float4(dB[0], dB[1], dB[2], dB[3]);
            *reinterpret_cast<float4*>(&sm.bc[t][kk][NS + 4 * l]) = make_float4(dC[0], dC[1], dC[2], dC[3]);
        };
        if (s0 < tb) {  // no sequence starts in the tile
#pragma unroll
            for (int t = 0; t < TT - 1; ++t) forward(t);
            backward(TT - 1, std::false_type{});
#pragma unroll
            for (int t = TT - 2; t >= 0; --t) backward(t, std::true_type{});
        } else {
            auto starts = [&](int64_t t, int& m) {  // whether token t is its sequence's first
                m = seq_of(p.cu, p.N, t);
                return (int64_t)p.cu[m] == t;
            };
            int m;
#pragma unroll
            for (int t = 0; t < TT; ++t) {
                if (t < nt && starts(tb + t, m)) {
                    if (t) load_tile(p.init, m, hs[t ? t - 1 : 0], 1.f);
                    else
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const int ch = c_lo + 4 * kk + i;
                            float4 f = make_float4(0.f, 0.f, 0.f, 0.f);
                            if (p.init && ch < c_hi)
                                f = *reinterpret_cast<const float4*>(p.init + ((int64_t)m * p.C + ch) * NS + 4 * l);
                            sm.ck[j & 1][i][tid] = f;
                        }
                }
                if (t < TT - 1) forward(t);
            }
#pragma unroll
            for (int t = TT - 1; t >= 0; --t) {
                backward(t, std::false_type{});
                if (t < nt && starts(tb + t, m)) {  // q is the initial state's gradient; on to the sequence before
                    if (b.dinit) store_tile(b.dinit, m, q);
                    if (tb + t > 0) {
                        n = seq_of(p.cu, p.N, tb + t - 1);
                        s0 = p.cu[n];
                        load_tile(b.dfin, n, q, 1.f);
                    }
                }
            }
        }
        cp_wait<0>();
        __syncthreads();

#pragma unroll
        for (int i = 0; i < PPT; ++i) {
            const int t = i * Y::RPT + row;
            if (t >= nt || !in0) continue;
            f2 s1 = f2_dup(0.f), s2 = s1, y = s1;
#pragma unroll
            for (int v = 0; v < L; ++v) {
                s1 = add2(s1, pair_of(&sm.part[0][t][v][cc]));
                s2 = add2(s2, pair_of(&sm.part[1][t][v][cc]));
                y = add2(y, pair_of(&sm.part[2][t][v][cc]));
            }
            // The elements come from shared memory once more: held since the step sizes they cost 16 registers (339 us
            // against 329 at 4,096 tokens x 4,096 channels x 16).
            const f2 d = pair_of(&sm.d[t][cc]), gv = pair_of(&sm.g[t][cc]), u = pair_of(&r.u[t][cc]);
            const int64_t o = (tb + t) * p.C + c0;
            store(b.du, o, fma2(d, s1, mul2(skip, gv)));
            f2 dd = fma2(u, s1, mul2(f2_dup(kLn2), s2));  // A2 carries log2 e
            if (p.softplus) dd = mul2(dd, sigmoid2(add2(pair_of(&r.dt[t][cc]), bias)));
            store(b.ddt, o, dd);
            accB = add2(accB, dd);
            accD = fma2(gv, u, accD);
            if (b.dz) {
                const f2 z = pair_of(&r.z[t][cc]), sg = sigmoid2(z), one = f2_dup(1.f);
                const f2 slope = mul2(sg, fma2(z, fma2(sg, f2_dup(-1.f), one), one));
                store(b.dz, o, mul2(mul2(pair_of(&r.dy[t][cc]), fma2(skip, u, y)), slope));
            }
        }
        // Two values of a token's row per thread, half of the parts in each half of a warp.
        float* pbc = b.pbc + ((int64_t)blockIdx.x * p.T + tb) * 2 * NS;
#pragma unroll
        for (int i = warp * 16 + lane % 16; i < TT * NS; i += NT / 2) {
            const int t = i / NS, v = 2 * (i % NS);
            f2 s = f2_dup(0.f);
#pragma unroll
            for (int k = 0; k < Y::KK; k += 2) s = add2(s, pair_of(&sm.bc[t][k + lane / 16][v]));
            s = add2(s, f2_of(__shfl_xor_sync(0xffffffffu, f2_lo(s), 16), __shfl_xor_sync(0xffffffffu, f2_hi(s), 16)));
            if (t < nt && lane < 16) put2(pbc + 2 * i, s);
        }
        // d and g of this tile are read above, and written again only by the same thread's next tile
    }
    store_tile(b.pa, piece, dA);
    if (row < Y::RPC) {
        float* o = b.pd + ((int64_t)piece * Y::RPC + row) * 2 * p.C + c0;
        if (in0) o[0] = f2_lo(accD), o[p.C] = f2_lo(accB);
        if (in1) o[1] = f2_hi(accD), o[p.C + 1] = f2_hi(accB);
    }
}

// dB and dC: the sums over a group's blocks.
template <typename T>
__global__ void __launch_bounds__(256) k_bc_sum(const float* __restrict__ part, int64_t T_total, int G, int bpg, int NS,
                                                T* __restrict__ dB, T* __restrict__ dC) {
    const int64_t W = T_total * 2 * NS, i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i >= W) return;
    const int g = blockIdx.y;
    float s = 0.f;
#pragma unroll 8
    for (int k = 0; k < bpg; ++k) s += part[((int64_t)g * bpg + k) * W + i];
    const int64_t t = i / (2 * NS), v = i % (2 * NS);
    T* o = v < NS ? dB : dC;
    o[(t * G + g) * NS + v % NS] = from_f<T>(s);
}

struct PutRow {
    float* p;
    __device__ void operator()(int64_t c, float s) const { p[c] = s; }
};
struct PutDB {  // column c of [dD | ddt_bias]
    float *dd, *db;
    int C;
    __device__ void operator()(int64_t c, float s) const {
        if (c < C) {
            if (dd) dd[c] = s;
        } else if (db) {
            db[c - C] = s;
        }
    }
};

int rpc_of(int ns) { return ns <= 32 ? ns / 8 : 4; }
int ch_of(int ns) { return 2048 / ns; }

template <typename T, int NS>
cudaError_t backward_as(BParams& b, const kda_ssm_backward_args& a, cudaStream_t s) {
    using Y = BLay<NS>;
    Params& p = b.f;
    cudaError_t e;
    if ((e = launch_states(p, a.fwd, s))) return e;
    if (p.pieces > 1) {
        constexpr int CB = Lay<NS, 1>::CB;
        k_rev<T, NS><<<dim3((unsigned)((p.Cg + CB - 1) / CB * p.G), p.pieces - 1), Lay<NS, 1>::NT, 0, s>>>(b);
        if ((e = cudaGetLastError())) return e;
        if (p.pieces > 2) {
            k_rev_join<NS><<<(unsigned)(((int64_t)p.C * NS + kJoinThreads - 1) / kJoinThreads), kJoinThreads, 0, s>>>(b);
            if ((e = cudaGetLastError())) return e;
        }
    }
    const int smem = (int)sizeof(BShared<T, NS>);
    if ((e = cudaFuncSetAttribute(k_ssm_bwd<T, NS>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem))) return e;
    k_ssm_bwd<T, NS><<<dim3((unsigned)(b.bpg * p.G), p.pieces), Y::NT, smem, s>>>(b);
    if ((e = cudaGetLastError())) return e;
    const int64_t W = p.T * 2 * NS;
    k_bc_sum<T><<<dim3((unsigned)((W + 255) / 256), p.G), 256, 0, s>>>(b.pbc, p.T, p.G, b.bpg, NS, static_cast<T*>(a.dB),
                                                                       static_cast<T*>(a.dC));
    if ((e = cudaGetLastError())) return e;
    if ((e = launch_column_sum(b.pa, p.pieces, (int64_t)p.C * NS, PutRow{a.dA}, s))) return e;
    if (!a.dD && !a.ddt_bias) return cudaSuccess;
    return launch_column_sum(b.pd, (int64_t)p.pieces * Y::RPC, 2 * (int64_t)p.C, PutDB{a.dD, a.ddt_bias, p.C}, s);
}

}  // namespace

SsmBackwardPlan ssm_backward_plan(const kda_ssm_args& f) {
    DeviceInfo di{0, 0, 0};
    const int64_t sms = current_device_info(&di) ? di.sm_count : 1;
    const int64_t cg = f.C / f.G, ch = ch_of(f.Nst), blocks = f.G * ((cg + ch - 1) / ch);
    SsmBackwardPlan p{};
    // Two blocks of the main kernel run on an SM and eight of the passes before it, of which there are up to twice as
    // many: two whole rounds of the former are one of the latter (4,096 tokens x 4,096 channels x 16: 0.67 ms for forward
    // and gradients, 0.75, 0.71 and 0.70 with one, three and four rounds).  Pieces of at least 64 tokens.
    int64_t k = 4 * sms / blocks;
    if (k > kMaxPieces) k = kMaxPieces;
    if (k > f.T_total / 64) k = f.T_total / 64;
    if (k < 1) k = 1;
    p.piece = ((f.T_total + k - 1) / k + 7) / 8 * 8;
    p.pieces = (int)((f.T_total + p.piece - 1) / p.piece);
    const size_t st = (size_t)f.C * f.Nst * sizeof(float), row = (size_t)f.C * sizeof(float);
    size_t at = 0;
    auto take = [&at](size_t bytes) {
        const size_t o = at;
        at += (bytes + 255) / 256 * 256;
        return o;
    };
    p.fwd = take(p.pieces * st);
    p.rev = take(p.pieces * st);
    p.fsum = take(p.pieces * row);
    p.rsum = take(p.pieces * row);
    p.ckpt = take((size_t)(f.T_total + 3) / 4 * st);
    p.pa = take(p.pieces * st);
    p.pd = take((size_t)p.pieces * rpc_of(f.Nst) * 2 * row);
    p.pbc = take((size_t)blocks * f.T_total * 2 * f.Nst * sizeof(float));
    p.workspace = at;
    return p;
}

cudaError_t launch_ssm_backward(const kda_ssm_backward_args& a, const SsmBackwardPlan& pl, cudaStream_t s) {
    BParams b{};
    b.f = params_of(a.fwd);
    char* ws = static_cast<char*>(a.workspace);
    auto at = [ws](size_t o) { return reinterpret_cast<float*>(ws + o); };
    b.f.piece = pl.piece;
    b.f.pieces = pl.pieces;
    b.f.ws_state = at(pl.fwd);
    b.f.ws_sum = at(pl.fsum);
    b.f.ckpt = at(pl.ckpt);
    b.f.fin = nullptr;
    b.rev = at(pl.rev);
    b.rsum = at(pl.rsum);
    b.pa = at(pl.pa);
    b.pd = at(pl.pd);
    b.pbc = at(pl.pbc);
    b.dy = a.dy;
    b.dys = a.dy_stride ? a.dy_stride : a.fwd.C;
    b.dfin = a.d_final_state;
    b.dinit = a.dinitial_state;
    b.du = a.du;
    b.ddt = a.ddt;
    b.dz = a.fwd.z ? a.dz : nullptr;
    const int es = a.fwd.io == KDA_BF16 ? 2 : 4, ch = ch_of(a.fwd.Nst);
    b.bpg = (b.f.Cg + ch - 1) / ch;
    auto pairs = [es](const void* q) { return reinterpret_cast<uintptr_t>(q) % (2 * es) == 0; };
    b.wide = b.f.Cg % 2 == 0 && pairs(b.du) && pairs(b.ddt) && pairs(b.dz);
    b.vec = b.f.vec && reinterpret_cast<uintptr_t>(a.dy) % 16 == 0 && b.dys * es % 16 == 0 &&
            b.dys * es < (int64_t)1 << 32;
#define KDA_BWD(T)                                               \
    switch (a.fwd.Nst) {                                         \
        case 8: return backward_as<T, 8>(b, a, s);               \
        case 16: return backward_as<T, 16>(b, a, s);             \
        case 32: return backward_as<T, 32>(b, a, s);             \
        default: return backward_as<T, 64>(b, a, s);             \
    }
    if (a.fwd.io == KDA_BF16) { KDA_BWD(bf16) } else { KDA_BWD(float) }
#undef KDA_BWD
}

}  // namespace kda
