// kda_ssm_scan.cu -- the selective state space scan: packed prompts and one token per sequence.
//
//   delta = softplus(dt + b),  h_t[n] = 2^(delta A[n] log2 e) h_{t-1}[n] + delta u B_t[n],
//   y_t = (sum_n C_t[n] h_t[n] + D u) silu(z)
//
// Per (token, channel, state) one exponential and four multiply-add-pipe operations (one of them 2^x's
// argument), against 8 / N bytes of HBM traffic: at N = 16 the arithmetic weighs more than the bytes (8,192
// tokens of 12,288 channels: 0.17 ms of either pipe, 0.12 ms of HBM).  So a thread keeps all (up to 16)
// states and decay rates of its channels in registers as pairs (fp32x2 instructions), and nothing but the
// token's B and C (fp32 in shared memory, one broadcast read for all lanes) and its step size comes from
// outside.  Rows come in tiles of eight tokens by asynchronous copies, three tiles in flight.
//
// One channel's tokens are a chain, and channels alone do not fill the GPU: the token axis is cut into
// pieces.  kPiece runs every piece from a zero state, k_scan_join carries the states through (a piece's
// effect on what enters it is 2^(A log2 e sum of delta)), kOut runs the pieces again from the right states.
//
// A decay 2^(delta A log2 e) carries the hardware exponential's 4 units of 2^-24 and 2 |delta A| of its exponent's
// roundings; correcting the exponent as the step size's (softplus2) would put two more instructions on every pair of
// states, in a loop that is nothing else.
//
// Measured, 8,192 x 12,288 x 16 bf16 with the gate: 695 us = 406 (kOut, 2.0 TB/s) + 280 (kPiece) + 9.
// Bound by latency at low occupancy: 17 to 20 % of an SM's warps (168 and 128 registers), which issue in 58 to 63 %
// of the cycles and wait for their own paired instructions (two or three cycles each) first; the exponential unit is
// 49 to 62 % busy.  Taken out one at a time in a copy of 488 us, the exponentials were worth 35 us, reading B
// and C 56, softplus 50, the gate 40, the copies 67, the stores 0.
//
// Sequences are walked, not mapped: a piece of the packed stream starts in the middle of whatever
// sequence holds its first token, and at a border the state is stored and the next one's loaded.
// kPiece begins at the last sequence that starts in its piece: nothing before it leaves the piece (8,192 tokens in
// sequences of 512: 275 -> 199 us, of 128: 70, when the step was made).
#include "kda_ssm.cuh"

namespace kda {

namespace {

using namespace ssm;

// kOut: the outputs, from the carried state.  kPiece: the state that a piece leaves when it starts
// from zero (or from the initial state of a sequence that starts at its first token or inside it; what
// lies before the last of them is passed over), and its sum of delta.  kStates: from the carried state, the state in front of every fourth token.
enum { kPiece, kOut, kStates };

// Channels per thread: two, so that a token's B and C are read from shared memory once for both (8,192 tokens x
// 12,288 channels x 16: outputs 455 -> 403 us, six blocks of 168 registers per SM against eight of 128); one for the
// checkpoints, whose stores of two rows per thread cost more than that (4,096 x 4,096 x 16: 73 against 93 us).
template <int NS, int kMode> using ScanLay = Lay<NS, kMode == kStates ? 1 : 2>;
// A value per channel of a thread: a pair, or one.
template <int CPT> struct Chans {
    using V = f2;
};
template <> struct Chans<1> {
    using V = float;
};
__device__ __forceinline__ float chan(f2 v, int k) { return k ? f2_hi(v) : f2_lo(v); }
__device__ __forceinline__ float chan(float v, int) { return v; }
__device__ __forceinline__ f2 times(f2 a, f2 b) { return mul2(a, b); }
__device__ __forceinline__ float times(float a, float b) { return a * b; }
__device__ __forceinline__ f2 plus(f2 a, f2 b) { return add2(a, b); }
__device__ __forceinline__ float plus(float a, float b) { return a + b; }
__device__ __forceinline__ void join_chans(f2& v, float a, float b) { v = f2_of(a, b); }
__device__ __forceinline__ void join_chans(float& v, float a, float) { v = a; }

template <typename T, int NS, int kMode>
__global__ void __launch_bounds__(ScanLay<NS, kMode>::NT, kMode == kOut ? 6 : 8) k_scan(Params p) {
    using Y = ScanLay<NS, kMode>;
    constexpr bool kMain = kMode == kOut;
    constexpr int CPT = Y::CPT;
    using V = typename Chans<CPT>::V;
    constexpr int L = Y::L, TT = Y::TT, NT = Y::NT, BPT = Y::BPT, H = Y::SPT / 2, Q = Y::SPT / 4, CB = Y::CB;
    constexpr int kDepth = 3;  // tiles in flight (four: no gain)
    struct Tile {
        T u[TT][CB], dt[TT][CB], z[kMain ? TT : 1][CB], B[TT][NS], C[kMain ? TT : 1][NS];
    };
    __shared__ __align__(16) Tile ring[kDepth];
    __shared__ __align__(16) float sB[2][TT][NS], sC[kMain ? 2 : 1][TT][NS];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int l = lane / Y::KPW;  // which SPT states of the channel
    const int bpg = (p.Cg + CB - 1) / CB, g = blockIdx.x / bpg;  // blocks per group
    const int c_lo = g * p.Cg + (blockIdx.x % bpg) * CB, c_hi = (g + 1) * p.Cg, cols = c_hi - c_lo;
    const int cl = CPT * (warp * Y::KPW + lane % Y::KPW), ch = c_lo + cl;  // this thread's (first) channel
    const bool gate = kMain && p.z;
    auto in = [&](int k) { return ch + k < c_hi; };  // threads past the group shadow its last channel, store nothing
    const int piece = blockIdx.y;
    const int64_t t0 = piece * p.piece, t1 = t0 + p.piece < p.T ? t0 + p.piece : p.T;
    uint32_t so[CPT];  // this thread's states in a row of [C][NS]
    f2 A2[CPT][H], h[CPT][H];
    V bias, skip, dsum;
#pragma unroll
    for (int k = 0; k < CPT; ++k) {
        const int c = in(k) ? ch + k : c_hi - 1;
        so[k] = (uint32_t)(c * NS + l * Y::SPT);
#pragma unroll
        for (int i = 0; i < Q; ++i) {
            const float4 a = __ldg(reinterpret_cast<const float4*>(p.A + so[k]) + i);
            A2[k][2 * i] = f2_of(a.x * kLog2e, a.y * kLog2e);
            A2[k][2 * i + 1] = f2_of(a.z * kLog2e, a.w * kLog2e);
        }
    }
    auto both = [&](const float* v) {  // a parameter of this thread's channels
        V o;
        join_chans(o, v && in(0) ? v[ch] : 0.f, CPT == 2 && v && in(1) ? v[ch + 1] : 0.f);
        return o;
    };
    bias = both(p.dt_bias);
    skip = both(kMain ? p.D : nullptr);
    dsum = both(nullptr);
    auto load_state = [&](const float* base, int64_t n) {  // row n of [..][C][NS], or zeros
#pragma unroll
        for (int k = 0; k < CPT; ++k)
#pragma unroll
            for (int i = 0; i < Q; ++i) {
                float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
                if (base) s = reinterpret_cast<const float4*>(base + n * p.C * NS + so[k])[i];
                h[k][2 * i] = f2_of(s.x, s.y);
                h[k][2 * i + 1] = f2_of(s.z, s.w);
            }
    };
    auto store_state = [&](float* base, int64_t n) {
#pragma unroll
        for (int k = 0; k < CPT; ++k)
            if (in(k))
#pragma unroll
                for (int i = 0; i < Q; ++i)
                    reinterpret_cast<float4*>(base + n * p.C * NS + so[k])[i] =
                        make_float4(f2_lo(h[k][2 * i]), f2_hi(h[k][2 * i]), f2_lo(h[k][2 * i + 1]), f2_hi(h[k][2 * i + 1]));
    };
    T* yp = static_cast<T*>(p.y) + ch + t0 * p.ys;
    const int tiles = (int)((t1 - t0 + TT - 1) / TT);
    auto issue = [&](int k) {  // copies of tile k (a group of its own, empty past the end)
        if (k < tiles) {
            Tile& r = ring[k % kDepth];
            const int64_t tb = t0 + (int64_t)k * TT;
            const int rows = (int)(t1 - tb < TT ? t1 - tb : TT);
            const uint32_t row = (uint32_t)tb;
            copy_tile<T, TT, CB, NT>(&r.u[0][0], static_cast<const T*>(p.u) + c_lo, p.us, row, rows, cols, p.vec);
            copy_tile<T, TT, CB, NT>(&r.dt[0][0], static_cast<const T*>(p.dt) + c_lo, p.dts, row, rows, cols, p.vec);
            if (gate)
                copy_tile<T, TT, CB, NT>(&r.z[0][0], static_cast<const T*>(p.z) + c_lo, p.zs, row, rows, cols, p.vec);
            copy_tile<T, TT, NS, NT>(&r.B[0][0], static_cast<const T*>(p.B) + g * NS, p.bs, row, rows, NS, p.vec);
            if (kMain)
                copy_tile<T, TT, NS, NT>(&r.C[0][0], static_cast<const T*>(p.Cm) + g * NS, p.cs, row, rows, NS, p.vec);
        }
        cp_commit();
    };
    auto widen = [&](int k) {  // B and C of tile k in fp32
        const Tile& r = ring[k % kDepth];
#pragma unroll
        for (int j = 0; j < BPT; ++j) {
            const int i = j * NT + tid;
            sB[k & 1][i / NS][i % NS] = to_f(r.B[i / NS][i % NS]);
            if (kMain) sC[k & 1][i / NS][i % NS] = to_f(r.C[i / NS][i % NS]);
        }
    };
#pragma unroll
    for (int k = 0; k < kDepth - 1; ++k) issue(k);
    int first = 0;  // tile
    if (kMode == kPiece) {  // the sequence that goes on behind the piece is all that leaves a state: up to it
        const int64_t s = p.cu[seq_of(p.cu, p.N, t1 - 1)];
        if (s >= t0 + TT) {
            first = (int)((s - t0) / TT < tiles - 1 ? (s - t0) / TT : tiles - 1);
            cp_wait<0>();  // those copies are not wanted
            __syncthreads();
#pragma unroll
            for (int k = 0; k < kDepth - 1; ++k) issue(first + k);
        }
    }
    int n = seq_of(p.cu, p.N, t0 + first * TT);
    int64_t seq_end = p.cu[n + 1];
    if (p.cu[n] == t0 + first * TT) load_state(p.init, n);
    else if (kMode != kPiece && piece > 0) load_state(p.ws_state, piece);
    else load_state(nullptr, 0);
    cp_wait<kDepth - 2>();  // the first tile
    __syncthreads();
    widen(first);
    for (int k = first; k < tiles; ++k) {
        const int64_t tb = t0 + (int64_t)k * TT;
        const int buf = k & 1;
        cp_wait<kDepth - 3>();  // tile k + 1
        __syncthreads();        // its rows are visible, tile k's fp32 rows too, and tile k - 1 is done with
        if (k + 1 < tiles) widen(k + 1);
        issue(k + kDepth - 1);
        const Tile& r = ring[k % kDepth];
        const int nt = (int)(t1 - tb < TT ? t1 - tb : TT);
        // One token: the states move on; the return value is this thread's part of sum_n C h.
        auto token = [&](int t, V d, V u) {
            const V x = times(d, u);
            f2 y[CPT];
#pragma unroll
            for (int k = 0; k < CPT; ++k) y[k] = f2_dup(0.f);
#pragma unroll
            for (int i = 0; i < Q; ++i) {
                const float4 b = *reinterpret_cast<const float4*>(&sB[buf][t][l * Y::SPT + 4 * i]);
                // the product first, then the multiply-add that shares du: three different register pairs in one
                // instruction cost a third cycle
#pragma unroll
                for (int k = 0; k < CPT; ++k) {
                    const f2 dd = f2_dup(chan(d, k)), du = f2_dup(chan(x, k));
                    h[k][2 * i] = fma2(du, f2_of(b.x, b.y), mul2(exp2_2(mul2(dd, A2[k][2 * i])), h[k][2 * i]));
                    h[k][2 * i + 1] = fma2(du, f2_of(b.z, b.w), mul2(exp2_2(mul2(dd, A2[k][2 * i + 1])), h[k][2 * i + 1]));
                }
                if (kMain) {
                    const float4 v = *reinterpret_cast<const float4*>(&sC[buf][t][l * Y::SPT + 4 * i]);
#pragma unroll
                    for (int k = 0; k < CPT; ++k) {
                        y[k] = fma2(h[k][2 * i], f2_of(v.x, v.y), y[k]);
                        y[k] = fma2(h[k][2 * i + 1], f2_of(v.z, v.w), y[k]);
                    }
                }
            }
            if (!kMain) dsum = plus(dsum, d);
            V out;
            join_chans(out, f2_lo(y[0]) + f2_hi(y[0]), f2_lo(y[CPT - 1]) + f2_hi(y[CPT - 1]));
            return out;
        };
        auto soft = [&](f2 x) { return p.softplus ? softplus2(x) : x; };
        auto finish = [&](int t, V y, V u) {  // the parts of a channel, the skip, the gate
            if constexpr (kMain) {
#pragma unroll
                for (int o = Y::KPW; o < 32; o *= 2)
                    y = add2(y, f2_of(__shfl_xor_sync(0xffffffffu, f2_lo(y), o), __shfl_xor_sync(0xffffffffu, f2_hi(y), o)));
                y = fma2(skip, u, y);
                if (gate) {
                    const f2 z = pair_of(&r.z[t][cl]);
                    y = mul2(y, mul2(z, sigmoid2(z)));
                }
            }
            return y;
        };
        auto put = [&](V y) {  // a row's outputs, and on to the next row
            if constexpr (kMain) {
                if (in(0) && (L == 1 || l == 0)) {
                    if (p.wide) {
                        put2(yp, y);
                    } else {
                        yp[0] = from_f<T>(f2_lo(y));
                        if (in(1)) yp[1] = from_f<T>(f2_hi(y));
                    }
                }
                yp += p.ys;
            }
        };
        if (nt == TT && seq_end >= tb + TT) {  // no border: eight tokens without a branch between them
            V d[TT], u[TT], y[TT];
            if constexpr (CPT == 2) {
#pragma unroll
                for (int t = 0; t < TT; ++t) {
                    d[t] = soft(add2(pair_of(&r.dt[t][cl]), bias));
                    u[t] = pair_of(&r.u[t][cl]);
                }
            } else {
#pragma unroll
                for (int t = 0; t < TT; t += 2) {
                    const f2 v = soft(add2(f2_of(to_f(r.dt[t][cl]), to_f(r.dt[t + 1][cl])), f2_dup(bias)));
                    d[t] = f2_lo(v);
                    d[t + 1] = f2_hi(v);
                    u[t] = to_f(r.u[t][cl]);
                    u[t + 1] = to_f(r.u[t + 1][cl]);
                }
            }
#pragma unroll
            for (int t = 0; t < TT; ++t) {
                if (kMode == kStates && t % 4 == 0) store_state(p.ckpt, (tb + t) / 4);
                y[t] = token(t, d[t], u[t]);
            }
#pragma unroll
            for (int t = 0; t < TT; ++t) y[t] = finish(t, y[t], u[t]);
#pragma unroll
            for (int t = 0; t < TT; ++t) put(y[t]);
        } else {
#pragma unroll 1
            for (int t = 0; t < nt; ++t) {
                if (kMode == kStates && t % 4 == 0) store_state(p.ckpt, (tb + t) / 4);
                if (tb + t == seq_end) {  // sequence n ended before this token
                    if (kMain && p.fin) store_state(p.fin, n);
                    while (n < p.N - 1 && p.cu[n + 1] <= tb + t) ++n;
                    seq_end = p.cu[n + 1];
                    load_state(p.init, n);
                }
                V d, u;
                if constexpr (CPT == 2) {
                    d = soft(add2(pair_of(&r.dt[t][cl]), bias));
                    u = pair_of(&r.u[t][cl]);
                } else {
                    d = f2_lo(soft(f2_dup(to_f(r.dt[t][cl]) + bias)));
                    u = to_f(r.u[t][cl]);
                }
                put(finish(t, token(t, d, u), u));
            }
        }
    }
    if (kMain) {
        if (p.fin && seq_end == t1) store_state(p.fin, n);
    } else if (kMode == kPiece) {
        store_state(p.ws_state, piece + 1);
        if (l == 0)
#pragma unroll
            for (int k = 0; k < CPT; ++k)
                if (in(k)) p.ws_sum[(int64_t)piece * p.C + ch + k] = chan(dsum, k);
    }
}

// The state at each piece's start, in the slots where the pieces left their own: slot k + 1 holds what
// piece k leaves by itself, and then what piece k + 1 starts from.
template <int NS> __global__ void __launch_bounds__(kJoinThreads) k_scan_join(Params p) {
    __shared__ uint32_t closed[kJoinBits / 32];
    mark_closed<1>(p, closed);
    const int64_t i = (int64_t)blockIdx.x * kJoinThreads + threadIdx.x, row = (int64_t)p.C * NS;
    if (i >= row) return;
    const float a2 = p.A[i] * kLog2e;
    float* slot = p.ws_state + row + i;  // of piece 0
    join<1>(p, closed, 1, p.pieces - 2, a2, *slot, slot, p.ws_sum + i / NS, row);
}

// One token per sequence: a thread holds 4 states of one channel and takes several sequences in turn,
// kRows states in flight at once.  Bound by HBM: the state read and written.  kVec: a thread's four
// elements of B and C come in one access.
// 256 sequences x 12,288 channels x 16, bf16: 76 us (5.6 TB/s); fp32 95 us (4.8 TB/s, 28 bytes spilled per thread).
constexpr int kStepThreads = 256;
constexpr int kRows = 4;
template <typename T, int NS, bool kVec> __global__ void __launch_bounds__(kStepThreads, 3) k_step(Params p, int rows) {
    constexpr int L = NS / 4, W = kVec ? 4 : 1;
    const int64_t i = (int64_t)blockIdx.x * kStepThreads + threadIdx.x;
    const int l = (int)(i % L);
    const bool in = i / L < p.C;
    const int64_t c = in ? i / L : p.C - 1;  // idle threads shadow the last channel and store nothing
    const int64_t g = c / p.Cg;
    const float4 a = *reinterpret_cast<const float4*>(p.A + c * NS + 4 * l);
    const f2 a2[2] = {f2_of(a.x * kLog2e, a.y * kLog2e), f2_of(a.z * kLog2e, a.w * kLog2e)};
    const float bias = p.dt_bias ? p.dt_bias[c] : 0.f, skip = p.D ? p.D[c] : 0.f;
    const T *up = static_cast<const T*>(p.u) + c, *dp = static_cast<const T*>(p.dt) + c;
    const T* zp = p.z ? static_cast<const T*>(p.z) + c : nullptr;
    const T *bp = static_cast<const T*>(p.B) + g * NS + 4 * l, *cp = static_cast<const T*>(p.Cm) + g * NS + 4 * l;
    float* sp = p.fin + c * NS + 4 * l;
    // Row r of a tensor: 32 x 32 bits to 64 in one instruction (row strides are below 4 GB).
    auto at = [](auto* base, uint32_t r, uint32_t bytes) {
        return reinterpret_cast<decltype(base)>(reinterpret_cast<uintptr_t>(base) + (uint64_t)r * bytes);
    };
    const uint32_t ub = (uint32_t)p.us * sizeof(T), db = (uint32_t)p.dts * sizeof(T), zb = (uint32_t)p.zs * sizeof(T),
                   bb = (uint32_t)p.bs * sizeof(T), cb = (uint32_t)p.cs * sizeof(T), yb = (uint32_t)p.ys * sizeof(T),
                   sb = (uint32_t)p.C * NS * sizeof(float);
    const int first = blockIdx.y * rows, last = first + rows < p.N ? first + rows : p.N;  // this block's sequences
    auto val = [](const Raw<T, 1>& r) {
        float v[1];
        unraw(r, v);
        return v[0];
    };
    auto four = [](const Raw<T, W> (&r)[4 / W], f2 (&o)[2]) {
        float v[4];
#pragma unroll
        for (int j = 0; j < 4 / W; ++j) {
            float t[W];
            unraw(r[j], t);
#pragma unroll
            for (int k = 0; k < W; ++k) v[j * W + k] = t[k];
        }
        o[0] = f2_of(v[0], v[1]);
        o[1] = f2_of(v[2], v[3]);
    };
    for (int r0 = first; r0 < last; r0 += kRows) {
        const int n = last - r0;  // sequences left
        float4 s[kRows];
        Raw<T, 1> u[kRows], x[kRows], z[kRows];
        Raw<T, W> b[kRows][4 / W], cc[kRows][4 / W];
#pragma unroll
        for (int q = 0; q < kRows; ++q) {
            const uint32_t r = r0 + (q < n ? q : 0);
            s[q] = in ? *at(reinterpret_cast<const float4*>(sp), r, sb) : make_float4(0.f, 0.f, 0.f, 0.f);
            u[q].load(at(up, r, ub));
            x[q].load(at(dp, r, db));
            if (zp) z[q].load(at(zp, r, zb));
#pragma unroll
            for (int j = 0; j < 4 / W; ++j) {
                b[q][j].load(at(bp, r, bb) + j * W);
                cc[q][j].load(at(cp, r, cb) + j * W);
            }
        }
#pragma unroll
        for (int q = 0; q < kRows; ++q) {
            if (q >= n) break;  // the same for the whole block
            const float uv = val(u[q]), xv = val(x[q]) + bias, d = p.softplus ? softplus(xv) : xv;
            const f2 dd = f2_dup(d), du = f2_dup(d * uv);
            f2 bv[2], cv[2];
            four(b[q], bv);
            four(cc[q], cv);
            const f2 h0 = fma2(exp2_2(mul2(dd, a2[0])), f2_of(s[q].x, s[q].y), mul2(du, bv[0]));
            const f2 h1 = fma2(exp2_2(mul2(dd, a2[1])), f2_of(s[q].z, s[q].w), mul2(du, bv[1]));
            const f2 y2 = fma2(h1, cv[1], mul2(h0, cv[0]));
            float y = f2_lo(y2) + f2_hi(y2);
#pragma unroll
            for (int o = 1; o < L; o *= 2) y += __shfl_xor_sync(0xffffffffu, y, o);
            if (in) {
                *at(reinterpret_cast<float4*>(sp), r0 + q, sb) = make_float4(f2_lo(h0), f2_hi(h0), f2_lo(h1), f2_hi(h1));
                y = fmaf(skip, uv, y);
                if (l == 0) *at(static_cast<T*>(p.y) + c, r0 + q, yb) = from_f<T>(zp ? y * silu(val(z[q])) : y);
            }
        }
    }
}

// The states at the pieces' starts, then the pass over all pieces.
template <typename T, int NS, int kMode> cudaError_t scan_as(const Params& p, cudaStream_t s) {
    // Blocks of a pass: those of the channels times `pieces`.
    auto grid = [&p](int cb, int pieces) { return dim3((unsigned)((p.Cg + cb - 1) / cb * p.G), (unsigned)pieces); };
    if (p.pieces > 1) {
        k_scan<T, NS, kPiece><<<grid(ScanLay<NS, kPiece>::CB, p.pieces - 1), ScanLay<NS, kPiece>::NT, 0, s>>>(p);
        if (cudaError_t e = cudaGetLastError()) return e;
        if (p.pieces > 2) {
            k_scan_join<NS><<<(unsigned)(((int64_t)p.C * NS + kJoinThreads - 1) / kJoinThreads), kJoinThreads, 0, s>>>(p);
            if (cudaError_t e = cudaGetLastError()) return e;
        }
    }
    k_scan<T, NS, kMode><<<grid(ScanLay<NS, kMode>::CB, p.pieces), ScanLay<NS, kMode>::NT, 0, s>>>(p);
    return cudaGetLastError();
}

template <int kMode> cudaError_t scan_mode(const Params& p, const kda_ssm_args& a, cudaStream_t s) {
#define KDA_SCAN(T)                                              \
    switch (a.Nst) {                                             \
        case 8: return scan_as<T, 8, kMode>(p, s);               \
        case 16: return scan_as<T, 16, kMode>(p, s);             \
        case 32: return scan_as<T, 32, kMode>(p, s);             \
        default: return scan_as<T, 64, kMode>(p, s);             \
    }
    if (a.io == KDA_BF16) { KDA_SCAN(bf16) } else { KDA_SCAN(float) }
#undef KDA_SCAN
}

template <typename T, int NS> cudaError_t step_as(const Params& p, cudaStream_t s) {
    const int64_t threads = (int64_t)p.C * (NS / 4);
    // Sequences per thread: four at once, and more rounds (up to four) while three blocks per SM are left.
    DeviceInfo di{0, 0, 0};
    const int64_t blocks = (threads + kStepThreads - 1) / kStepThreads, sms = current_device_info(&di) ? di.sm_count : 1;
    int rows = kRows;
    while (rows < 4 * kRows && blocks * ((p.N + 2 * rows - 1) / (2 * rows)) >= 3 * sms) rows *= 2;
    while ((p.N + rows - 1) / rows > 65535) rows *= 2;
    const dim3 g((unsigned)blocks, (unsigned)((p.N + rows - 1) / rows));
    constexpr int bytes = 4 * sizeof(T);
    auto wide = [](const void* q, int64_t stride) {
        return reinterpret_cast<uintptr_t>(q) % bytes == 0 && stride * sizeof(T) % bytes == 0;
    };
    if (wide(p.B, p.bs) && wide(p.Cm, p.cs)) k_step<T, NS, true><<<g, kStepThreads, 0, s>>>(p, rows);
    else k_step<T, NS, false><<<g, kStepThreads, 0, s>>>(p, rows);
    return cudaGetLastError();
}

}  // namespace

ssm::Params ssm::params_of(const kda_ssm_args& a) {
    auto or_ = [](int64_t s, int64_t d) { return s ? s : d; };
    Params p{};
    const int64_t gn = (int64_t)a.G * a.Nst;
    p.u = a.u; p.dt = a.dt; p.z = a.z; p.B = a.B; p.Cm = a.Cm; p.y = a.y;
    p.us = or_(a.u_stride, a.C); p.dts = or_(a.dt_stride, a.C); p.zs = or_(a.z_stride, a.C);
    p.bs = or_(a.B_stride, gn); p.cs = or_(a.C_stride, gn); p.ys = or_(a.y_stride, a.C);
    p.A = a.A; p.D = a.D; p.dt_bias = a.dt_bias; p.init = a.initial_state; p.fin = a.final_state;
    p.cu = a.cu_seqlens;
    p.T = a.T_total; p.N = a.N; p.C = a.C; p.G = a.G; p.Cg = a.C / a.G;
    p.softplus = a.softplus;
    const int es = a.io == KDA_BF16 ? 2 : 4;
    auto wide = [es](const void* q, int64_t stride) {
        return reinterpret_cast<uintptr_t>(q) % 16 == 0 && stride * es % 16 == 0 && stride * es < (int64_t)1 << 32;
    };
    p.vec = wide(p.u, p.us) && wide(p.dt, p.dts) && (!p.z || wide(p.z, p.zs)) && wide(p.B, p.bs) && wide(p.Cm, p.cs) &&
            (int64_t)p.Cg * es % 16 == 0;
    p.wide = p.Cg % 2 == 0 && p.ys % 2 == 0 && reinterpret_cast<uintptr_t>(p.y) % (2 * es) == 0;
    return p;
}

ScanPlan scan_plan(const kda_ssm_args& a) {
    DeviceInfo di{0, 0, 0};
    const int64_t sms = current_device_info(&di) ? di.sm_count : 1;
    const int64_t tt = 8, cb = a.Nst <= 16 ? 128 : 2048 / a.Nst;  // ScanLay<Nst, kOut>'s tile and channels per block
    ScanPlan p{};
    const int64_t blocks = a.G * ((a.C / a.G + cb - 1) / cb);
    // Two whole rounds of blocks, of which six run on an SM (five in fp32 with 8 or 16 states, whose rings take 39 to
    // 42 KB: 2.4 rounds there); pieces of at least 8 tiles.  (One piece of 8,192
    // tokens x 12,288 channels leaves most warp slots empty: 1.5 ms, against 0.69 ms in 19 pieces, the pass over
    // their own states included; one round: 0.76 ms, three: 0.71, four: 0.69.)
    int64_t k = 12 * sms / blocks;
    if (k > kMaxPieces) k = kMaxPieces;
    const int64_t most = a.T_total / (8 * tt);
    if (k > most) k = most;
    if (k < 1) k = 1;
    p.piece = ((a.T_total + k - 1) / k + tt - 1) / tt * tt;
    if (p.piece < tt) p.piece = tt;
    p.pieces = (int)((a.T_total + p.piece - 1) / p.piece);
    if (p.pieces > 1) {
        p.sums = (size_t)p.pieces * a.C * a.Nst * sizeof(float);
        p.workspace = p.sums + (size_t)p.pieces * a.C * sizeof(float);
    }
    return p;
}

cudaError_t launch_ssm_scan(const kda_ssm_args& a, const ScanPlan& pl, cudaStream_t s) {
    Params p = params_of(a);
    p.piece = pl.piece;
    p.pieces = pl.pieces;
    p.ws_state = static_cast<float*>(a.workspace);
    p.ws_sum = reinterpret_cast<float*>(static_cast<char*>(a.workspace) + pl.sums);
    return scan_mode<kOut>(p, a, s);
}

cudaError_t ssm::launch_states(const Params& p, const kda_ssm_args& a, cudaStream_t s) { return scan_mode<kStates>(p, a, s); }

cudaError_t launch_ssm_step(const kda_ssm_args& a, cudaStream_t s) {
    const Params p = params_of(a);
#define KDA_STEP(T)                                              \
    switch (a.Nst) {                                             \
        case 8: return step_as<T, 8>(p, s);                      \
        case 16: return step_as<T, 16>(p, s);                    \
        case 32: return step_as<T, 32>(p, s);                    \
        default: return step_as<T, 64>(p, s);                    \
    }
    if (a.io == KDA_BF16) { KDA_STEP(bf16) } else { KDA_STEP(float) }
#undef KDA_STEP
}

}  // namespace kda
