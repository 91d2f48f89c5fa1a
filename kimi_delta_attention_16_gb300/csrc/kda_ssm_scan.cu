// kda_ssm_scan.cu -- the selective state space scan: packed prompts and one token per sequence.
//
//   delta = softplus(dt + b),  h_t[n] = 2^(delta A[n] log2 e) h_{t-1}[n] + delta u B_t[n],
//   y_t = (sum_n C_t[n] h_t[n] + D u) silu(z)
//
// Per (token, channel, state) one exponential and four multiply-add-pipe operations, against 8 / N
// bytes of HBM traffic per state: at N = 16 the arithmetic weighs more than the bytes (8,192 tokens
// of 12,288 channels: 0.17 ms of either pipe, 0.12 ms of HBM).  So the inner loop keeps states and
// decay rates in registers as pairs (fp32x2 instructions), reads a token's B and C once for two
// channels, and leaves each thread's part of y in shared memory, where the epilogue adds the parts
// of a channel, the skip and the gate.  Tokens come in tiles: the next tile's loads are in flight
// while the current one is scanned.
//
// Sequences are walked, not mapped: a piece of the packed stream starts in the middle of whatever
// sequence holds its first token, and at a border the state is stored and the next one's loaded.
#include "kda_ssm.cuh"

namespace kda {

namespace {

using namespace ssm;

// kMain: the outputs.  Otherwise the state that a piece leaves when it starts from zero (or from the
// initial state of a sequence that starts at its first token or inside it), and its sum of delta.
template <typename T, int NS, bool kMain>
__global__ void __launch_bounds__(Lay<NS>::kThreads) k_scan(Params p) {
    using Y = Lay<NS>;
    constexpr int L = Y::L, TT = Y::TT, NT = Y::kThreads, EPT = Y::EPT, BPT = Y::BPT;
    __shared__ float2 sd[TT][kCB];                            // delta, delta u
    __shared__ __align__(16) float sB[TT][NS], sC[kMain ? TT : 1][NS];
    __shared__ __align__(16) float sy[kMain ? TT : 1][kCB][L];  // parts of sum_n C h
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int g = blockIdx.x / p.bpg;
    const int c_lo = g * p.Cg + (blockIdx.x % p.bpg) * kCB, c_hi = (g + 1) * p.Cg;
    const int piece = blockIdx.y;
    const int64_t t0 = piece * p.piece, t1 = t0 + p.piece < p.T ? t0 + p.piece : p.T;

    // this thread's states: channels cp and cp + 32 of the block, states 4 l .. 4 l + 3
    const int l = lane / Y::KPW, cp = warp * Y::KPW + lane % Y::KPW;
    const int ch[2] = {c_lo + cp, c_lo + cp + 32};
    f2 A2[2][2], h[2][2];
    float dsum[2] = {0.f, 0.f};
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
        if (ch[i] < c_hi) a = *reinterpret_cast<const float4*>(p.A + (int64_t)ch[i] * NS + 4 * l);
        A2[i][0] = f2_of(a.x * kLog2e, a.y * kLog2e);
        A2[i][1] = f2_of(a.z * kLog2e, a.w * kLog2e);
    }
    auto load_state = [&](const float* base, int64_t n) {  // row n of [..][C][NS], or zeros
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
            if (base && ch[i] < c_hi) s = *reinterpret_cast<const float4*>(base + (n * p.C + ch[i]) * NS + 4 * l);
            h[i][0] = f2_of(s.x, s.y);
            h[i][1] = f2_of(s.z, s.w);
        }
    };
    auto store_state = [&](float* base, int64_t n) {
#pragma unroll
        for (int i = 0; i < 2; ++i)
            if (ch[i] < c_hi)
                *reinterpret_cast<float4*>(base + (n * p.C + ch[i]) * NS + 4 * l) =
                    make_float4(f2_lo(h[i][0]), f2_hi(h[i][0]), f2_lo(h[i][1]), f2_hi(h[i][1]));
    };
    int n = seq_of(p.cu, p.N, t0);
    int64_t seq_end = p.cu[n + 1];
    if (p.cu[n] == t0) load_state(p.init, n);
    else if (kMain && piece > 0) load_state(p.ws_state, piece);
    else load_state(nullptr, 0);
    auto cross = [&](int64_t t) {  // sequence n ended before token t
        if (kMain && p.fin) store_state(p.fin, n);
        while (n < p.N - 1 && p.cu[n + 1] <= t) ++n;
        seq_end = p.cu[n + 1];
        load_state(p.init, n);
    };

    // this thread's elements of a tile: tokens tid / kCB + k (NT / kCB), one channel
    const int ec = c_lo + tid % kCB, et = tid / kCB;
    const bool ein = ec < c_hi;
    const float bias = ein && p.dt_bias ? p.dt_bias[ec] : 0.f;
    const float skip = kMain && ein && p.D ? p.D[ec] : 0.f;
    const T* up = static_cast<const T*>(p.u) + ec;
    const T* dp = static_cast<const T*>(p.dt) + ec;
    const T* zp = kMain && p.z ? static_cast<const T*>(p.z) + ec : nullptr;
    const T* bp = static_cast<const T*>(p.B) + (int64_t)g * NS;
    const T* cpn = static_cast<const T*>(p.Cm) + (int64_t)g * NS;
    Raw<T, 1> ru[EPT], rd[EPT], rz[EPT], rb[BPT], rc[BPT];
    auto fetch = [&](int64_t tb) {
#pragma unroll
        for (int k = 0; k < EPT; ++k) {
            const int64_t t = tb + et + k * (NT / kCB);
            ru[k].zero(); rd[k].zero(); rz[k].zero();
            if (t < t1 && ein) {
                ru[k].load(up + t * p.us);
                rd[k].load(dp + t * p.dts);
                if (zp) rz[k].load(zp + t * p.zs);
            }
        }
#pragma unroll
        for (int k = 0; k < BPT; ++k) {
            const int i = k * NT + tid;
            const int64_t t = tb + i / NS;
            rb[k].zero(); rc[k].zero();
            if (t < t1) {
                rb[k].load(bp + t * p.bs + i % NS);
                if (kMain) rc[k].load(cpn + t * p.cs + i % NS);
            }
        }
    };
    fetch(t0);
    for (int64_t tb = t0; tb < t1; tb += TT) {
        float u[EPT], z[EPT];
#pragma unroll
        for (int k = 0; k < EPT; ++k) {
            float v[1];
            unraw(ru[k], v);
            u[k] = v[0];
            unraw(rz[k], v);
            z[k] = v[0];
            unraw(rd[k], v);
            const float x = v[0] + bias;
            float d = p.softplus ? softplus(x) : x;
            if (tb + et + k * (NT / kCB) >= t1 || !ein) d = 0.f;
            sd[et + k * (NT / kCB)][tid % kCB] = make_float2(d, d * u[k]);
        }
#pragma unroll
        for (int k = 0; k < BPT; ++k) {
            const int i = k * NT + tid;
            float v[1];
            unraw(rb[k], v);
            sB[i / NS][i % NS] = v[0];
            if (kMain) {
                unraw(rc[k], v);
                sC[i / NS][i % NS] = v[0];
            }
        }
        __syncthreads();
        if (tb + TT < t1) fetch(tb + TT);

        auto token = [&](int t) {
            const float4 b = *reinterpret_cast<const float4*>(&sB[t][4 * l]);
            const f2 b0 = f2_of(b.x, b.y), b1 = f2_of(b.z, b.w);
            f2 c0, c1;
            if (kMain) {
                const float4 c = *reinterpret_cast<const float4*>(&sC[t][4 * l]);
                c0 = f2_of(c.x, c.y);
                c1 = f2_of(c.z, c.w);
            }
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const float2 dv = sd[t][cp + 32 * i];
                const f2 d = f2_dup(dv.x), du = f2_dup(dv.y);
                h[i][0] = fma2(exp2_2(mul2(d, A2[i][0])), h[i][0], mul2(du, b0));
                h[i][1] = fma2(exp2_2(mul2(d, A2[i][1])), h[i][1], mul2(du, b1));
                if (kMain) {
                    const f2 y = fma2(h[i][1], c1, mul2(h[i][0], c0));
                    sy[t][cp + 32 * i][l] = f2_lo(y) + f2_hi(y);
                } else {
                    dsum[i] += dv.x;
                }
            }
        };
        if (tb == seq_end) cross(tb);
        if (tb + TT <= t1 && seq_end >= tb + TT) {
#pragma unroll 4
            for (int t = 0; t < TT; ++t) token(t);
        } else {
            const int nt = (int)(t1 - tb < TT ? t1 - tb : TT);
#pragma unroll 1
            for (int t = 0; t < nt; ++t) {
                if (tb + t == seq_end) cross(tb + t);
                token(t);
            }
        }
        __syncthreads();
        if (kMain && ein) {
            T* yp = static_cast<T*>(p.y) + ec;
#pragma unroll
            for (int k = 0; k < EPT; ++k) {
                const int t = et + k * (NT / kCB);
                if (tb + t >= t1) continue;
                float s = skip * u[k];
#pragma unroll
                for (int j = 0; j < L; ++j) s += sy[t][tid % kCB][j];
                yp[(tb + t) * p.ys] = from_f<T>(p.z ? s * silu(z[k]) : s);
            }
        }
    }
    if (kMain) {
        if (p.fin && seq_end == t1) store_state(p.fin, n);
    } else {
        store_state(p.ws_state, piece + 1);
        if (l == 0)
#pragma unroll
            for (int i = 0; i < 2; ++i)
                if (ch[i] < c_hi) p.ws_sum[(int64_t)piece * p.C + ch[i]] = dsum[i];
    }
}

// The state at each piece's start, in the slots where the pieces left their own: carried state
// times 2^(A log2 e sum of delta), unless a sequence started in the piece, plus the piece's own.
template <int NS> __global__ void __launch_bounds__(256) k_scan_join(Params p) {
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x, row = (int64_t)p.C * NS;
    if (i >= row) return;
    const int64_t c = i / NS;
    const float a2 = p.A[i] * kLog2e;
    float carry = p.ws_state[row + i];
#pragma unroll 4
    for (int k = 1; k < p.pieces - 1; ++k) {
        const int64_t t1 = (k + 1) * p.piece;
        const bool started = p.cu[seq_of(p.cu, p.N, t1 - 1)] >= k * p.piece;
        const float own = p.ws_state[(k + 1) * row + i];
        const float f = exp2_hw(a2 * p.ws_sum[(int64_t)k * p.C + c]);
        carry = started ? own : fmaf(f, carry, own);
        p.ws_state[(k + 1) * row + i] = carry;
    }
}

// One token per sequence: a thread holds 4 states of one channel and takes several sequences in
// turn, kRows states in flight at once.  Bound by HBM: the state read and written.
constexpr int kStepThreads = 256;
constexpr int kRows = 4;
template <typename T, int NS> __global__ void __launch_bounds__(kStepThreads) k_step(Params p) {
    constexpr int L = NS / 4;
    const int64_t i = (int64_t)blockIdx.x * kStepThreads + threadIdx.x;
    const int l = (int)(i % L);
    const bool in = i / L < p.C;
    const int64_t c = in ? i / L : p.C - 1;  // idle threads shadow the last channel and store nothing
    const int64_t g = c / p.Cg;
    const float4 a = *reinterpret_cast<const float4*>(p.A + c * NS + 4 * l);
    const float a2[4] = {a.x * kLog2e, a.y * kLog2e, a.z * kLog2e, a.w * kLog2e};
    const float bias = p.dt_bias ? p.dt_bias[c] : 0.f, skip = p.D ? p.D[c] : 0.f;
    const T *up = static_cast<const T*>(p.u) + c, *dp = static_cast<const T*>(p.dt) + c;
    const T* zp = p.z ? static_cast<const T*>(p.z) + c : nullptr;
    const T *bp = static_cast<const T*>(p.B) + g * NS + 4 * l, *cp = static_cast<const T*>(p.Cm) + g * NS + 4 * l;
    T* yp = static_cast<T*>(p.y) + c;
    for (int64_t r0 = (int64_t)blockIdx.y * kRows; r0 < p.N; r0 += (int64_t)gridDim.y * kRows) {
        float4 s[kRows];
        float u[kRows], x[kRows], z[kRows], b[kRows][4], cc[kRows][4];
#pragma unroll
        for (int q = 0; q < kRows; ++q) {
            const int64_t r = r0 + q < p.N ? r0 + q : p.N - 1;
            s[q] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (in) s[q] = *reinterpret_cast<const float4*>(p.fin + (r * p.C + c) * NS + 4 * l);
            u[q] = ldf(up + r * p.us);
            x[q] = ldf(dp + r * p.dts) + bias;
            z[q] = zp ? ldf(zp + r * p.zs) : 0.f;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                b[q][j] = ldf(bp + r * p.bs + j);
                cc[q][j] = ldf(cp + r * p.cs + j);
            }
        }
#pragma unroll
        for (int q = 0; q < kRows; ++q) {
            const float d = p.softplus ? softplus(x[q]) : x[q], du = d * u[q];
            float h[4] = {s[q].x, s[q].y, s[q].z, s[q].w}, y = 0.f;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                h[j] = fmaf(exp2_hw(d * a2[j]), h[j], du * b[q][j]);
                y = fmaf(h[j], cc[q][j], y);
            }
#pragma unroll
            for (int o = 1; o < L; o *= 2) y += __shfl_xor_sync(0xffffffffu, y, o);
            const int64_t r = r0 + q;
            if (r >= p.N || !in) continue;
            *reinterpret_cast<float4*>(p.fin + (r * p.C + c) * NS + 4 * l) = make_float4(h[0], h[1], h[2], h[3]);
            y = fmaf(skip, u[q], y);
            if (l == 0) yp[r * p.ys] = from_f<T>(zp ? y * silu(z[q]) : y);
        }
    }
}

int64_t or_(int64_t s, int64_t d) { return s ? s : d; }

Params params_of(const kda_ssm_args& a) {
    Params p{};
    const int64_t gn = (int64_t)a.G * a.Nst;
    p.u = a.u; p.dt = a.dt; p.z = a.z; p.B = a.B; p.Cm = a.Cm; p.y = a.y;
    p.us = or_(a.u_stride, a.C); p.dts = or_(a.dt_stride, a.C); p.zs = or_(a.z_stride, a.C);
    p.bs = or_(a.B_stride, gn); p.cs = or_(a.C_stride, gn); p.ys = or_(a.y_stride, a.C);
    p.A = a.A; p.D = a.D; p.dt_bias = a.dt_bias; p.init = a.initial_state; p.fin = a.final_state;
    p.cu = a.cu_seqlens;
    p.T = a.T_total; p.N = a.N; p.C = a.C; p.G = a.G; p.Cg = a.C / a.G;
    p.bpg = (p.Cg + kCB - 1) / kCB;
    p.softplus = a.softplus;
    return p;
}

template <typename T, int NS> cudaError_t scan_as(const Params& p, cudaStream_t s) {
    const int nt = Lay<NS>::kThreads;
    const unsigned gx = (unsigned)(p.bpg * p.G);
    if (p.pieces > 1) {
        k_scan<T, NS, false><<<dim3(gx, p.pieces - 1), nt, 0, s>>>(p);
        if (cudaError_t e = cudaGetLastError()) return e;
        if (p.pieces > 2) {
            k_scan_join<NS><<<(unsigned)(((int64_t)p.C * NS + 255) / 256), 256, 0, s>>>(p);
            if (cudaError_t e = cudaGetLastError()) return e;
        }
    }
    k_scan<T, NS, true><<<dim3(gx, p.pieces), nt, 0, s>>>(p);
    return cudaGetLastError();
}

template <typename T, int NS> cudaError_t step_as(const Params& p, cudaStream_t s) {
    const int64_t threads = (int64_t)p.C * (NS / 4);
    const int64_t rows = (p.N + kRows - 1) / kRows;
    k_step<T, NS><<<dim3((unsigned)((threads + kStepThreads - 1) / kStepThreads), (unsigned)(rows < 65535 ? rows : 65535)),
                    kStepThreads, 0, s>>>(p);
    return cudaGetLastError();
}

}  // namespace

ScanPlan scan_plan(const kda_ssm_args& a) {
    DeviceInfo di{0, 0, 0};
    const int64_t sms = current_device_info(&di) ? di.sm_count : 1;
    const int64_t cg = a.C / a.G, blocks = a.G * ((cg + kCB - 1) / kCB);
    const int64_t warps = blocks * (a.Nst / 4), tt = a.Nst == 64 ? 8 : 16;
    ScanPlan p{};
    // Enough warps for 16 per SM, pieces of at least 8 tiles.
    int64_t k = (16 * sms + warps - 1) / warps;
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
#define KDA_SCAN(T)                                              \
    switch (a.Nst) {                                             \
        case 8: return scan_as<T, 8>(p, s);                      \
        case 16: return scan_as<T, 16>(p, s);                    \
        case 32: return scan_as<T, 32>(p, s);                    \
        default: return scan_as<T, 64>(p, s);                    \
    }
    if (a.io == KDA_BF16) { KDA_SCAN(bf16) } else { KDA_SCAN(float) }
#undef KDA_SCAN
}

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
