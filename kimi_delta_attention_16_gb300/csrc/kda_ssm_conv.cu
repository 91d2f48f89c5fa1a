// kda_ssm_conv.cu -- the selective scan's causal depthwise convolution of width 4: packed prompts,
// one token per sequence, and the gradients.
//
//   pre_t = bias + sum_j w[j] x[t-3+j],  y_t = silu(pre_t)
//   dpre_t = dy_t silu'(pre_t),  dx_t = sum_j w[j] dpre_{t+3-j},  dw[j] = sum_t dpre_t x[t-3+j]
//
// Bound by HBM (one read of x, one write of y; backward: x and dy read, dx written).  A thread
// owns kWide = 4 consecutive channels (one element where the layout allows no more) and walks a run of
// tokens with the last three raw values in registers; its rows come by asynchronous copies into a ring of
// its own in shared memory, up to four batches of kBatch tokens ahead (batches loaded to registers kept
// too few bytes in flight: forward 60 -> 48 us, backward 128 -> 97).
// The backward walks forward too: the contributions to the last three dx wait in registers, and a run
// reads three tokens past its end to finish its own.  dw and dbias: per thread over its run, per block over
// its runs through shared memory, then over the blocks, in a fixed order.
//
// Measured, 8,192 x 8,192 bf16 in 7 sequences: forward 46 us (5.8 TB/s), backward 97 us (4.2 TB/s: two blocks
// of 128-register threads per SM); one token for 256 sequences of 12,288 channels 12 us.
#include "kda_block.cuh"

namespace kda {

namespace {

constexpr int kThreads = 256;
constexpr int kBatch = 4;  // tokens taken together
constexpr int kWide = 4;  // channels per thread where the layout allows (8 bytes of bf16, 16 of fp32)

// A thread's own rows (W channels, consecutive tokens) through shared memory: up to four batches of kBatch
// tokens are in flight, the thread reads back what it copied itself, so nothing waits for anybody else.
// Accesses below 4 bytes (bf16 rows that allow no more) cannot be copied this way: those are read when
// their batch begins.
template <typename T, int W> struct Rows {
    static constexpr bool kAsync = Raw<T, W>::kBytes >= 4;
    static constexpr int kGroups = Raw<T, W>::kBytes == 16 ? 2 : 4;  // batches in flight: 128 bytes per thread
    static constexpr int kSlots = kAsync ? kGroups * kBatch : 1;
    Raw<T, W>* ring;  // [kSlots][kThreads], at this thread
    const T* src;     // the next token to copy
    int64_t stride;
    int left;         // tokens that are left to copy
    int next;         // slot of the next batch to copy
    Raw<T, W> now[kAsync ? 1 : kBatch];
    __device__ __forceinline__ void begin(Raw<T, W>* shared, const T* first, int64_t st, int tokens) {
        ring = shared + threadIdx.y * blockDim.x + threadIdx.x;
        src = first;
        stride = st;
        left = tokens;
        next = 0;
    }
    __device__ __forceinline__ void issue() {  // the caller commits
        if constexpr (kAsync) {
#pragma unroll
            for (int q = 0; q < kBatch; ++q) {
                if (q < left) cp_async_raw<T, W>(ring + (next + q) * kThreads, src);
                src += stride;
            }
            left -= kBatch;
            next = next + kBatch == kSlots ? 0 : next + kBatch;
        }
    }
    __device__ __forceinline__ void take() {  // the batch at the front, where it is read now
        if constexpr (!kAsync) {
#pragma unroll
            for (int q = 0; q < kBatch; ++q) {
                if (q < left) now[q].load(src);
                src += stride;
            }
            left -= kBatch;
        }
    }
    // Token q of the batch in slots [slot, slot + kBatch).
    __device__ __forceinline__ Raw<T, W> get(int slot, int q) const {
        if constexpr (kAsync) return ring[(slot + q) * kThreads];
        Raw<T, W> r = now[0];
#pragma unroll
        for (int k = 1; k < (kAsync ? 1 : kBatch); ++k)
            if (q == k) r = now[k];
        return r;
    }
};

// Raw value at place `pos` (< 0: before the sequence, from the conv state or zero), W channels from c.
template <typename T, int W>
__device__ __forceinline__ void place(const T* __restrict__ x, int64_t xs, const T* __restrict__ cs, int64_t s, int64_t pos,
                                      int64_t n, int C, int c, f2 (&v)[(W + 1) / 2]) {
    if (pos >= 0) {
        Raw<T, W> r;
        r.load(x + (s + pos) * xs + c);
        unraw2(r, v);
    } else {
        float t[W];
#pragma unroll
        for (int j = 0; j < W; ++j) t[j] = cs && pos >= -3 ? to_f(cs[(n * C + c + j) * 3 + 3 + pos]) : 0.f;
#pragma unroll
        for (int j = 0; j < (W + 1) / 2; ++j) v[j] = f2_of(t[2 * j], 2 * j + 1 < W ? t[2 * j + 1] : 0.f);
    }
}

// The three values before token t of a sequence that starts at s.  `raw` holds the three rows before t as
// they lie in memory (loaded before s was known); those before s come from the conv state instead.
template <typename T, int W>
__device__ __forceinline__ void window(const Raw<T, W> (&raw)[3], const T* __restrict__ x, int64_t xs, const T* __restrict__ cs,
                                       int64_t s, int64_t t, int64_t n, int C, int c, f2 (&win)[3][(W + 1) / 2]) {
#pragma unroll
    for (int m = 0; m < 3; ++m) {
        if (t - 3 + m >= s) unraw2(raw[m], win[m]);
        else place<T, W>(x, xs, cs, s, t - s - 3 + m, n, C, c, win[m]);
    }
}

// Taps and bias of W channels as pairs.
template <int W>
__device__ __forceinline__ void load_taps(const float* __restrict__ w, const float* __restrict__ bias, int64_t c,
                                          f2 (&wt)[4][(W + 1) / 2], f2 (&bs)[(W + 1) / 2]) {
#pragma unroll
    for (int j = 0; j < (W + 1) / 2; ++j) {
        const bool two = 2 * j + 1 < W;
#pragma unroll
        for (int k = 0; k < 4; ++k) wt[k][j] = f2_of(w[(c + 2 * j) * 4 + k], two ? w[(c + 2 * j + 1) * 4 + k] : 0.f);
        bs[j] = bias ? f2_of(bias[c + 2 * j], two ? bias[c + 2 * j + 1] : 0.f) : f2_dup(0.f);
    }
}

// W consecutive values of a state that the same kernel writes (no read-only cache).
template <int W> __device__ __forceinline__ void load_state(const float* p, float (&v)[W]) {
    if constexpr (W == 4) {
        const float4 f = *reinterpret_cast<const float4*>(p);
        v[0] = f.x; v[1] = f.y; v[2] = f.z; v[3] = f.w;
    } else {
        v[0] = *p;
    }
}
template <int W> __device__ __forceinline__ void load_state(const bf16* p, float (&v)[W]) {
    Raw<bf16, W> r;
    if constexpr (W == 4) {
        const uint2 u = *reinterpret_cast<const uint2*>(p);
        r.w[0] = u.x; r.w[1] = u.y;
    } else {
        r.w[0] = *reinterpret_cast<const unsigned short*>(p);
    }
    unraw(r, v);
}

template <typename T, int W>
__global__ void __launch_bounds__(kThreads, 2)
k_conv(const T* __restrict__ x, int64_t xs, const float* __restrict__ w, const float* __restrict__ bias, int silu,
       const int32_t* cu, int N, int64_t T_total, int C, const T* __restrict__ cs_in, T* __restrict__ cs_out,
       T* __restrict__ y, int64_t ys, int run, unsigned strips) {
    __shared__ int32_t staged[kStagedCu];
    __shared__ Raw<T, W> shared[Rows<T, W>::kSlots * kThreads];
    const unsigned rows = blockIdx.x / strips, strip = blockIdx.x - rows * strips;
    const int c = (strip * blockDim.x + threadIdx.x) * W;
    const int64_t t0 = ((int64_t)rows * blockDim.y + threadIdx.y) * run;
    const bool on = c < C && t0 < T_total;
    const int64_t t1 = t0 + run < T_total ? t0 + run : T_total;
    constexpr int P = (W + 1) / 2;
    Raw<T, W> before[3];
    f2 wt[4][P], bs[P], win[3][P];
    Rows<T, W> in;
    if (on) {
        in.begin(shared, x + t0 * xs + c, xs, (int)(t1 - t0));
#pragma unroll
        for (int g = 0; g < Rows<T, W>::kGroups - 1; ++g) {
            in.issue();
            cp_commit();
        }
#pragma unroll
        for (int m = 0; m < 3; ++m)
            if (t0 - 3 + m >= 0) before[m].load(x + (t0 - 3 + m) * xs + c);
        load_taps<W>(w, bias, c, wt, bs);
    }
    cu = stage_cu(cu, N, staged);
    if (!on) return;
    int n = seq_of(cu, N, t0);
    int64_t s, e;
    seq_range(cu, n, T_total, s, e);
    window<T, W>(before, x, xs, cs_in, s, t0, n, C, c, win);
    T* yp = y + t0 * ys + c;
    auto token = [&](const Raw<T, W>& raw) {
        f2 v[P], o[P];
        unraw2(raw, v);
#pragma unroll
        for (int j = 0; j < P; ++j) {
            o[j] = fma2(wt[3][j], v[j], fma2(wt[2][j], win[2][j], fma2(wt[1][j], win[1][j], fma2(wt[0][j], win[0][j], bs[j]))));
            if (silu) o[j] = mul2(o[j], sigmoid2(o[j]));
            win[0][j] = win[1][j];
            win[1][j] = win[2][j];
            win[2][j] = v[j];
        }
        store_row2<T, W>(yp, o);
        yp += ys;
    };
    int slot = 0;
    for (int64_t tb = t0; tb < t1; tb += kBatch) {
        in.issue();
        cp_commit();
        cp_wait<Rows<T, W>::kGroups - 1>();
        in.take();
        if (tb + kBatch <= t1 && tb + kBatch < e) {  // no sequence ends here: tokens without a branch between them
#pragma unroll
            for (int q = 0; q < kBatch; ++q) token(in.get(slot, q));
        } else
#pragma unroll 1
        for (int64_t t = tb; t < tb + kBatch && t < t1; ++t) {
            if (t >= e && n < N - 1) {  // crossed into a later sequence
                while (t >= e && n < N - 1) {
                    ++n;
                    seq_range(cu, n, T_total, s, e);
                }
#pragma unroll
                for (int m = 0; m < 3; ++m) place<T, W>(x, xs, cs_in, s, t - s - 3 + m, n, C, c, win[m]);
            }
            token(in.get(slot, (int)(t - tb)));
            if (cs_out && t == e - 1) {
#pragma unroll
                for (int j = 0; j < W; ++j)
#pragma unroll
                    for (int m = 0; m < 3; ++m)
                        cs_out[((int64_t)n * C + c + j) * 3 + m] = from_f<T>(j & 1 ? f2_hi(win[m][j / 2]) : f2_lo(win[m][j / 2]));
            }
        }
        slot = slot + kBatch >= Rows<T, W>::kSlots ? 0 : slot + kBatch;
    }
}

// One token per sequence: the three old values and the new one, the state rolled in place.  Its own
// thread reads and writes the state of W channels (3 W consecutive values: three accesses of W) and takes
// several sequences in turn, kStepRows of them in flight at once.
constexpr int kStepRows = 4;
template <typename T, int W>
__global__ void __launch_bounds__(kThreads)
k_conv_step(const T* __restrict__ x, int64_t xs, const float* __restrict__ w, const float* __restrict__ bias, int silu,
            int N, int C, T* cs, T* __restrict__ y, int64_t ys) {
    const int c = (blockIdx.x * kThreads + threadIdx.x) * W;
    if (c >= C) return;
    float wt[4][W], bs[W];
#pragma unroll
    for (int j = 0; j < W; ++j) {
#pragma unroll
        for (int k = 0; k < 4; ++k) wt[k][j] = w[(int64_t)(c + j) * 4 + k];
        bs[j] = bias ? bias[c + j] : 0.f;
    }
    for (int64_t n0 = (int64_t)blockIdx.y * kStepRows; n0 < N; n0 += (int64_t)gridDim.y * kStepRows) {
        float st[kStepRows][3 * W], xv[kStepRows][W];
#pragma unroll
        for (int q = 0; q < kStepRows; ++q) {
            const int64_t n = n0 + q < N ? n0 + q : N - 1;
            const T* p = cs + (n * C + c) * 3;
#pragma unroll
            for (int k = 0; k < 3; ++k) {
                float t[W];
                load_state(p + k * W, t);
#pragma unroll
                for (int j = 0; j < W; ++j) st[q][k * W + j] = t[j];
            }
            Raw<T, W> r;
            r.load(x + n * xs + c);
            unraw(r, xv[q]);
        }
#pragma unroll
        for (int q = 0; q < kStepRows; ++q) {
            const int64_t n = n0 + q;
            if (n >= N) break;
            float o[W], roll[3 * W];
#pragma unroll
            for (int j = 0; j < W; ++j) {
                float a = fmaf(wt[0][j], st[q][3 * j], bs[j]);
                a = fmaf(wt[1][j], st[q][3 * j + 1], a);
                a = fmaf(wt[2][j], st[q][3 * j + 2], a);
                a = fmaf(wt[3][j], xv[q][j], a);
                o[j] = silu ? a * sigmoid(a) : a;
                roll[3 * j] = st[q][3 * j + 1];
                roll[3 * j + 1] = st[q][3 * j + 2];
                roll[3 * j + 2] = xv[q][j];
            }
            store_row(y + n * ys + c, o);
            T* p = cs + (n * C + c) * 3;
#pragma unroll
            for (int k = 0; k < 3; ++k) {
                float t[W];
#pragma unroll
                for (int j = 0; j < W; ++j) t[j] = roll[k * W + j];
                store_row(p + k * W, t);
            }
        }
    }
}

template <typename T, int W>
__global__ void __launch_bounds__(kThreads, 2)
k_conv_bwd(const T* __restrict__ x, int64_t xs, const float* __restrict__ w, const float* __restrict__ bias, int silu,
           const int32_t* cu, int N, int64_t T_total, int C, const T* __restrict__ cs_in,
           const T* __restrict__ dy, int64_t dys, T* __restrict__ dx, int64_t dxs, float* __restrict__ dcs,
           float* __restrict__ part, int run, unsigned strips) {
    extern __shared__ __align__(16) float sm[];  // [blockDim.y][5][blockDim.x * W]
    __shared__ int32_t staged[kStagedCu];
    Raw<T, W>* shared_x = reinterpret_cast<Raw<T, W>*>(sm);  // the rows in flight; the sums of the block at the end
    Raw<T, W>* shared_d = shared_x + Rows<T, W>::kSlots * kThreads;
    const unsigned rows = blockIdx.x / strips, strip = blockIdx.x - rows * strips;
    const int c = (strip * blockDim.x + threadIdx.x) * W;
    const int64_t t0 = ((int64_t)rows * blockDim.y + threadIdx.y) * run;
    const int64_t t1 = t0 + run < T_total ? t0 + run : T_total, last = t1 + 3 < T_total ? t1 + 3 : T_total;
    constexpr int P = (W + 1) / 2;
    f2 gw[5][P];  // dw[0..3], dbias
#pragma unroll
    for (int k = 0; k < 5; ++k)
#pragma unroll
        for (int j = 0; j < P; ++j) gw[k][j] = f2_dup(0.f);
    Raw<T, W> before[3];
    f2 wt[4][P], bs[P];
    const bool on = c < C && t0 < T_total;
    Rows<T, W> inx, ind;
    if (on) {
        inx.begin(shared_x, x + t0 * xs + c, xs, (int)(last - t0));
        ind.begin(shared_d, dy + t0 * dys + c, dys, (int)(last - t0));
#pragma unroll
        for (int g = 0; g < Rows<T, W>::kGroups - 1; ++g) {
            inx.issue();
            ind.issue();
            cp_commit();
        }
#pragma unroll
        for (int m = 0; m < 3; ++m)
            if (t0 - 3 + m >= 0) before[m].load(x + (t0 - 3 + m) * xs + c);
        load_taps<W>(w, bias, c, wt, bs);
    }
    cu = stage_cu(cu, N, staged);
    if (on) {
        f2 win[3][P], pend[3][P], out[P];
#pragma unroll
        for (int j = 0; j < P; ++j) pend[0][j] = pend[1][j] = pend[2][j] = f2_dup(0.f);
        int n = seq_of(cu, N, t0);
        int64_t s, e;
        seq_range(cu, n, T_total, s, e);
        window<T, W>(before, x, xs, cs_in, s, t0, n, C, c, win);
        // The finished gradient of the value at place p (absolute): a token of this run, or one of the
        // three values before a sequence that starts in it.
        auto put = [&](int64_t p, const f2 (&v)[P]) {
            if (p >= s) {
                if (p >= t0 && p < t1) store_row2<T, W>(dx + p * dxs + c, v);
            } else if (dcs && s >= t0 && p >= s - 3) {
#pragma unroll
                for (int j = 0; j < W; ++j)
                    dcs[((int64_t)n * C + c + j) * 3 + (p - s + 3)] = j & 1 ? f2_hi(v[j / 2]) : f2_lo(v[j / 2]);
            }
        };
        auto flush = [&](int64_t t) {  // the sequence ends before t: nothing more reaches the pending three
#pragma unroll
            for (int m = 0; m < 3; ++m) put(t - 3 + m, pend[m]);
        };
        bool open = true;  // the pending three still wait for tokens of their own sequence
        auto slope = [&](const f2 (&v)[P], f2 (&d)[P]) {  // dy of a token to dpre
            if (!silu) return;
#pragma unroll
            for (int j = 0; j < P; ++j) {
                const f2 a = fma2(wt[3][j], v[j],
                                  fma2(wt[2][j], win[2][j], fma2(wt[1][j], win[1][j], fma2(wt[0][j], win[0][j], bs[j]))));
                const f2 sg = sigmoid2(a), t = fma2(a, sub2(f2_dup(1.f), sg), f2_dup(1.f));
                d[j] = mul2(d[j], mul2(sg, t));
            }
        };
        auto sums = [&](const f2 (&v)[P], const f2 (&d)[P]) {
#pragma unroll
            for (int j = 0; j < P; ++j) {
                gw[0][j] = fma2(d[j], win[0][j], gw[0][j]);
                gw[1][j] = fma2(d[j], win[1][j], gw[1][j]);
                gw[2][j] = fma2(d[j], win[2][j], gw[2][j]);
                gw[3][j] = fma2(d[j], v[j], gw[3][j]);
                gw[4][j] = add2(gw[4][j], d[j]);
            }
        };
        auto move = [&](const f2 (&v)[P], const f2 (&d)[P]) {  // leaves the gradient of place t - 3 in `out`
#pragma unroll
            for (int j = 0; j < P; ++j) {
                win[0][j] = win[1][j];
                win[1][j] = win[2][j];
                win[2][j] = v[j];
                out[j] = fma2(wt[0][j], d[j], pend[0][j]);
                pend[0][j] = fma2(wt[1][j], d[j], pend[1][j]);
                pend[1][j] = fma2(wt[2][j], d[j], pend[2][j]);
                pend[2][j] = mul2(wt[3][j], d[j]);
            }
        };
        int slot = 0;
        for (int64_t tb = t0; tb < last && open; tb += kBatch) {
            inx.issue();
            ind.issue();
            cp_commit();
            cp_wait<Rows<T, W>::kGroups - 1>();
            inx.take();
            ind.take();
            const int at = slot;
            slot = slot + kBatch >= Rows<T, W>::kSlots ? 0 : slot + kBatch;
            if (tb - 3 >= t0 && tb - 3 >= s && tb + kBatch <= t1 && tb + kBatch <= e) {
                // own tokens only, and every finished place is one of them: no branch between the tokens
                T* op = dx + (tb - 3) * dxs + c;
#pragma unroll
                for (int q = 0; q < kBatch; ++q) {
                    f2 v[P], d[P];
                    unraw2(inx.get(at, q), v);
                    unraw2(ind.get(at, q), d);
                    slope(v, d);
                    sums(v, d);
                    move(v, d);
                    store_row2<T, W>(op, out);
                    op += dxs;
                }
                continue;
            }
#pragma unroll 1
            for (int64_t t = tb; t < tb + kBatch && t < last; ++t) {
                if (t >= e && n < N - 1) {
                    flush(e);
                    if (t >= t1) {  // past this run's tokens and its last sequence
                        open = false;
                        break;
                    }
                    while (t >= e && n < N - 1) {
                        ++n;
                        seq_range(cu, n, T_total, s, e);
                    }
#pragma unroll
                    for (int m = 0; m < 3; ++m) place<T, W>(x, xs, cs_in, s, t - s - 3 + m, n, C, c, win[m]);
#pragma unroll
                    for (int j = 0; j < P; ++j) pend[0][j] = pend[1][j] = pend[2][j] = f2_dup(0.f);
                }
                f2 v[P], d[P];
                unraw2(inx.get(at, (int)(t - tb)), v);
                unraw2(ind.get(at, (int)(t - tb)), d);
                slope(v, d);
                if (t < t1) sums(v, d);
                move(v, d);
                put(t - 3, out);
            }
        }
        if (open && last == T_total) flush(T_total);
    }
    const int bw = blockDim.x * W;  // channels of the block
    cp_wait<0>();
    __syncthreads();  // every thread is done with the rows that lie where the sums go
#pragma unroll
    for (int k = 0; k < 5; ++k)
#pragma unroll
        for (int j = 0; j < W; ++j) sm[(threadIdx.y * 5 + k) * bw + threadIdx.x * W + j] = j & 1 ? f2_hi(gw[k][j / 2]) : f2_lo(gw[k][j / 2]);
    __syncthreads();
    for (int i = threadIdx.y * blockDim.x + threadIdx.x; i < 5 * bw; i += blockDim.x * blockDim.y) {
        float t = 0.f;
        for (int r = 0; r < blockDim.y; ++r) t += sm[r * 5 * bw + i];
        const int k = i / bw, ch = strip * bw + i - k * bw;
        if (ch < C) part[((int64_t)rows * 5 + k) * C + ch] = t;
    }
}

struct PutConv {  // column k * C + c of [dw[0] | dw[1] | dw[2] | dw[3] | dbias]
    float *dw, *db;
    int C;
    __device__ void operator()(int64_t i, float s) const {
        const int64_t k = i / C, c = i - k * C;
        if (k < 4) {
            if (dw) dw[c * 4 + k] = s;
        } else if (db) {
            db[c] = s;
        }
    }
};

__global__ void k_empty_sequences(const int32_t* __restrict__ cu, int N, const uint16_t* __restrict__ src,
                                  uint16_t* __restrict__ dst, int64_t per) {
    for (int64_t n = blockIdx.y; n < N; n += gridDim.y) {
        if (cu[n + 1] != cu[n]) continue;
        for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < per; i += (int64_t)gridDim.x * blockDim.x)
            dst[n * per + i] = src ? src[n * per + i] : (uint16_t)0;
    }
}

bool wide(const void* p, int64_t stride, int es) {
    return reinterpret_cast<uintptr_t>(p) % (kWide * es) == 0 && stride % kWide == 0;
}
int64_t stride_or(int64_t s, int64_t d) { return s ? s : d; }

// Threads along the channels: a power of two, at most a warp.
int lanes_of(int accesses) {
    int x = 1;
    while (x < 32 && x < accesses) x *= 2;
    return x;
}

// Tokens per thread: long runs re-read fewer border tokens, short ones fill the GPU; 64 once
// there are over 1,024 threads per SM, never below 8.
int run_of(int64_t T, int64_t accesses) {
    DeviceInfo di{0, 0, 0};
    const int64_t want = 1024 * (int64_t)(current_device_info(&di) ? di.sm_count : 1);
    int run = 64;
    while (run > 8 && T * accesses / run < want) run /= 2;
    return run;
}

}  // namespace

cudaError_t launch_empty_sequences(const int32_t* cu, int N, const void* src, void* dst, int64_t per, cudaStream_t s) {
    const int64_t units = per / 2;
    const int64_t bx = (units + 255) / 256;
    k_empty_sequences<<<dim3((unsigned)(bx < 64 ? bx : 64), (unsigned)(N < 4096 ? N : 4096)), 256, 0, s>>>(
        cu, N, static_cast<const uint16_t*>(src), static_cast<uint16_t*>(dst), units);
    return cudaGetLastError();
}

cudaError_t launch_ssm_conv(const kda_ssm_conv_args& a, cudaStream_t s) {
    const int es = a.io == KDA_BF16 ? 2 : 4;
    const int64_t xs = stride_or(a.x_stride, a.C), ys = stride_or(a.y_stride, a.C);
    const bool vec = a.C % kWide == 0 && wide(a.x, xs, es) && wide(a.y, ys, es);
    const int W = vec ? kWide : 1;
    const int acc = (a.C + W - 1) / W;
    const dim3 b(lanes_of(acc), kThreads / lanes_of(acc));
    const int run = run_of(a.T_total, acc);
    // Blocks that run together cover whole rows (strips of channels first), not one strip of many rows.
    const unsigned strips = (unsigned)((acc + b.x - 1) / b.x);
    const unsigned g = strips * (unsigned)((a.T_total + (int64_t)run * b.y - 1) / ((int64_t)run * b.y));
#define KDA_CONV(T, W)                                                                                              \
    k_conv<T, W><<<g, b, 0, s>>>(static_cast<const T*>(a.x), xs, a.w, a.bias, a.silu, a.cu_seqlens, a.N, a.T_total,  \
                                 a.C, static_cast<const T*>(a.conv_state_in), static_cast<T*>(a.conv_state_out),     \
                                 static_cast<T*>(a.y), ys, run, strips)
    if (a.io == KDA_BF16) {
        if (vec) KDA_CONV(bf16, 4); else KDA_CONV(bf16, 1);
    } else {
        if (vec) KDA_CONV(float, 4); else KDA_CONV(float, 1);
    }
#undef KDA_CONV
    return cudaGetLastError();
}

cudaError_t launch_ssm_conv_step(const kda_ssm_conv_args& a, cudaStream_t s) {
    const int64_t xs = stride_or(a.x_stride, a.C), ys = stride_or(a.y_stride, a.C);
    const int es = a.io == KDA_BF16 ? 2 : 4;
    const bool vec = a.C % kWide == 0 && wide(a.x, xs, es) && wide(a.y, ys, es) && wide(a.conv_state_out, 0, es);
    const int W = vec ? kWide : 1, per = kThreads * W;
    const int64_t rows = (a.N + kStepRows - 1) / kStepRows;
    const dim3 g((unsigned)((a.C + per - 1) / per), (unsigned)(rows < 65535 ? rows : 65535));
#define KDA_CONVS(T, W)                                                                                             \
    k_conv_step<T, W><<<g, kThreads, 0, s>>>(static_cast<const T*>(a.x), xs, a.w, a.bias, a.silu, a.N, a.C,          \
                                             static_cast<T*>(a.conv_state_out), static_cast<T*>(a.y), ys)
    if (a.io == KDA_BF16) {
        if (vec) KDA_CONVS(bf16, 4); else KDA_CONVS(bf16, 1);
    } else {
        if (vec) KDA_CONVS(float, 4); else KDA_CONVS(float, 1);
    }
#undef KDA_CONVS
    return cudaGetLastError();
}

ConvBackwardPlan conv_backward_plan(const kda_ssm_conv_args& f) {
    // The layout of the rows may rule out wide accesses only after the workspace was sized, so the run
    // and the partial rows follow from sizes alone: those of the wide layout hold for both.
    const int acc = (f.C + kWide - 1) / kWide;
    ConvBackwardPlan p;
    p.run = run_of(f.T_total, acc);
    const int64_t by = kThreads / lanes_of(acc);
    p.rows = (f.T_total + p.run * by - 1) / (p.run * by);
    p.workspace = (size_t)p.rows * 5 * f.C * sizeof(float);
    return p;
}

cudaError_t launch_ssm_conv_backward(const kda_ssm_conv_backward_args& a, const ConvBackwardPlan& p, cudaStream_t s) {
    const kda_ssm_conv_args& f = a.fwd;
    const int es = f.io == KDA_BF16 ? 2 : 4;
    const int64_t xs = stride_or(f.x_stride, f.C), dys = stride_or(a.dy_stride, f.C), dxs = stride_or(a.dx_stride, f.C);
    const bool vec = f.C % kWide == 0 && wide(f.x, xs, es) && wide(a.dy, dys, es) && wide(a.dx, dxs, es);
    const int W = vec ? kWide : 1;
    const int lanes = lanes_of((f.C + kWide - 1) / kWide);
    const dim3 b(lanes, kThreads / lanes);
    const unsigned strips = (unsigned)((f.C + (int64_t)lanes * W - 1) / ((int64_t)lanes * W));
    const unsigned g = strips * (unsigned)p.rows;
    const size_t row = (size_t)2 * kThreads * (es * W == 16 ? 2 : 4) * kBatch * W * es, sum = (size_t)kThreads * 5 * W * sizeof(float);
    const int smem = (int)(row > sum ? row : sum);  // at most 64 KB
    cudaError_t e = cudaSuccess;
    float* part = static_cast<float*>(a.workspace);
#define KDA_CONVB(T, W)                                                                                             \
    if (!(e = cudaFuncSetAttribute(k_conv_bwd<T, W>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem)))            \
    k_conv_bwd<T, W><<<g, b, smem, s>>>(static_cast<const T*>(f.x), xs, f.w, f.bias, f.silu, f.cu_seqlens, f.N,      \
                                        f.T_total, f.C, static_cast<const T*>(f.conv_state_in),                      \
                                        static_cast<const T*>(a.dy), dys, static_cast<T*>(a.dx), dxs,                \
                                        a.dconv_state_in, part, p.run, strips)
    if (f.io == KDA_BF16) {
        if (vec) { KDA_CONVB(bf16, 4); } else { KDA_CONVB(bf16, 1); }
    } else {
        if (vec) { KDA_CONVB(float, 4); } else { KDA_CONVB(float, 1); }
    }
#undef KDA_CONVB
    if (!e) e = cudaGetLastError();
    if (e) return e;
    return launch_column_sum(part, p.rows, 5 * (int64_t)f.C, PutConv{a.dw, a.dbias, f.C}, s);
}

}  // namespace kda
