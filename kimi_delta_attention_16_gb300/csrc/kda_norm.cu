// kda_norm.cu -- layer norm over the last axis, forward and backward.
//
//   forward   mean, var = mean of squared deviations, y = (x - mean) rstd w + b
//   backward  xh = (x - mean) rstd, p = dy w:
//             dx = rstd (p - mean(p) - xh mean(p xh)),  dw = sum_rows dy xh,  db = sum_rows dy
//
// Both are bound by HBM: one read of x (and dy), one write of y (dx).  A row lives in the
// registers of one block (VPT accesses of W elements per thread), so the statistics take two
// passes over registers, none over memory: k_layer_norm, k_layer_norm_bwd.  Many rows in 16-byte layouts
// (k_layer_norm_rows, k_layer_norm_bwd_rows) are taken two at a time by persistent blocks, with
// the next ones on their way to a ring in shared memory: registers alone cannot hold enough
// loads in flight (8,192 x 7,168 bf16: forward 64 -> 40 us).  The backward is persistent: a thread owns the same
// columns in every row of its block, keeps their dw and db sums in registers and leaves one
// partial per block, which k_column_sum adds up in block order (no atomics: the same bits
// every time).
//
// Measured, 8,192 x 7,168 bf16: forward 40 us (5.8 TB/s), backward 70 us (5.0 TB/s; 75 from 8-bit x) and 6 us
// for the column sums.  The backward is bound by latency: 40 % of an SM's warps, one barrier and one chain of
// shuffles per row with one row in hand; its warps wait for memory and shared memory first, and 54 % of the issue
// slots are taken.  Rows wider than the ring kernels' (bf16 above 14,336 channels, fp32 above 7,168) keep dw and db of
// up to 32 channels per thread beside the row in 64 registers and spill, up to 2,000 bytes: 8,192 x 16,384 bf16 256 us
// (floor 119), fp32 986 (238).
#include "kda_block.cuh"

namespace kda {

namespace {

constexpr int kMaxWarps = 32;

// Sum over the block of one or two values; every thread gets it.  Two values share the shuffles: the
// first exchange leaves one of them in each half of the warp.  `buf` is written and read once: a caller
// that comes back to the same buffer has passed another barrier in between.
__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}
__device__ __forceinline__ float warp_sum2(float a, float b) {  // a's sum in the lower half, b's in the upper
    const bool up = threadIdx.x & 16;
    float v = (up ? b : a) + __shfl_xor_sync(0xffffffffu, up ? a : b, 16);
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}
template <int NT = 0> __device__ __forceinline__ void block_sum(float (&v)[1], float (*buf)[1]) {
    const int lane = threadIdx.x & 31, nw = (NT ? NT : blockDim.x) >> 5;
    v[0] = warp_sum(v[0]);
    if (nw == 1) return;
    if (lane == 0) buf[threadIdx.x >> 5][0] = v[0];
    __syncthreads();
    v[0] = warp_sum(lane < nw ? buf[lane][0] : 0.f);
}
template <int NT = 0> __device__ __forceinline__ void block_sum(float (&v)[2], float (*buf)[2]) {
    const int lane = threadIdx.x & 31, nw = (NT ? NT : blockDim.x) >> 5;
    float s = warp_sum2(v[0], v[1]);
    if (nw > 1) {
        if ((lane & 15) == 0) buf[threadIdx.x >> 5][lane >> 4] = s;
        __syncthreads();
        const float2 t = lane < nw ? *reinterpret_cast<const float2*>(buf[lane]) : make_float2(0.f, 0.f);
        s = warp_sum2(t.x, t.y);
    }
    v[0] = __shfl_sync(0xffffffffu, s, 0);
    v[1] = __shfl_sync(0xffffffffu, s, 16);
}

// Column of access i of this thread (in elements): consecutive threads take consecutive accesses.
template <int W, int NT = 0> __device__ __forceinline__ int col_of(int i) {  // NT: threads of the block, 0 when it varies
    return (i * (NT ? NT : (int)blockDim.x) + (int)threadIdx.x) * W;
}

template <typename T, int W, int VPT>
__global__ void __launch_bounds__(1024)
k_layer_norm(const T* __restrict__ x, int64_t xs, const float* __restrict__ w, const float* __restrict__ b, float eps,
             T* __restrict__ y, int64_t ys, float* __restrict__ stats, int64_t M, int C) {
    __shared__ float red[2][kMaxWarps][1];
    const float inv_c = 1.0f / (float)C;
    for (int64_t r = blockIdx.x; r < M; r += gridDim.x) {
        Raw<T, W> raw[VPT];
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int c = col_of<W>(i);
            if (c < C) raw[i].load(x + r * xs + c); else raw[i].zero();
        }
        float v[VPT][W], s[1] = {0.f};
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            unraw(raw[i], v[i]);
#pragma unroll
            for (int j = 0; j < W; ++j) s[0] += v[i][j];
        }
        block_sum(s, red[0]);
        const float mean = s[0] * inv_c;
        s[0] = 0.f;
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const bool in = col_of<W>(i) < C;
#pragma unroll
            for (int j = 0; j < W; ++j) {
                v[i][j] -= mean;
                if (in) s[0] = fmaf(v[i][j], v[i][j], s[0]);
            }
        }
        block_sum(s, red[1]);
        const float rstd = 1.0f / sqrtf(fmaf(s[0], inv_c, eps));
        if (stats && threadIdx.x == 0) {
            stats[2 * r] = mean;
            stats[2 * r + 1] = rstd;
        }
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int c = col_of<W>(i);
            if (c >= C) continue;
            float wv[W], bv[W];
            if (w) load_param(w + c, wv);
            if (b) load_param(b + c, bv);
#pragma unroll
            for (int j = 0; j < W; ++j) {
                const float n = v[i][j] * rstd;
                v[i][j] = w ? n * wv[j] : n;
                if (b) v[i][j] += bv[j];
            }
            store_row(y + r * ys + c, v[i]);
        }
    }
}

// ------------------------------------------------------------------ many rows
// Persistent blocks that take R rows at a time, with kDepth - 1 groups of them on their way to shared
// memory.  A thread copies and reads its own columns only, so no barrier guards the ring.  R = 2 rows
// share the shuffles and barriers of their sums, and arithmetic runs on fp32 pairs.
constexpr int kDepth = 3;

// Sums of four values over a warp: lane 0 gets a's, 16 b's, 8 c's, 24 d's (six shuffles).
__device__ __forceinline__ float warp_sum4(float a, float b, float c, float d) {
    const bool hi = threadIdx.x & 16, hi8 = threadIdx.x & 8;
    const float p = (hi ? b : a) + __shfl_xor_sync(0xffffffffu, hi ? a : b, 16);
    const float q = (hi ? d : c) + __shfl_xor_sync(0xffffffffu, hi ? c : d, 16);
    float v = (hi8 ? q : p) + __shfl_xor_sync(0xffffffffu, hi8 ? p : q, 8);
#pragma unroll
    for (int o = 4; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}
template <int NT> __device__ __forceinline__ void block_sum4(float (&v)[4], float (*buf)[4]) {
    const int lane = threadIdx.x & 31, nw = NT >> 5;
    float s = warp_sum4(v[0], v[1], v[2], v[3]);
    if (nw > 1) {
        if ((lane & 7) == 0) buf[threadIdx.x >> 5][((lane >> 4) & 1) + ((lane >> 2) & 2)] = s;
        __syncthreads();
        const float4 t = lane < nw ? *reinterpret_cast<const float4*>(buf[lane]) : make_float4(0.f, 0.f, 0.f, 0.f);
        s = warp_sum4(t.x, t.y, t.z, t.w);
    }
    v[0] = __shfl_sync(0xffffffffu, s, 0);
    v[1] = __shfl_sync(0xffffffffu, s, 16);
    v[2] = __shfl_sync(0xffffffffu, s, 8);
    v[3] = __shfl_sync(0xffffffffu, s, 24);
}
__device__ __forceinline__ float f2_sum(f2 v) { return f2_lo(v) + f2_hi(v); }

// Shapes of the row kernels: accesses per thread and threads, fixed so that every offset in the ring is a
// constant.  448 threads of 72 registers leave two blocks to an SM (7,168 bf16 channels: 2 x 448 accesses); up
// to 1,792 accesses take four per thread.  Wider rows go through the kernels above, one at a time.
constexpr int kRowThreads = 448;
constexpr int kRowAccesses = 4 * kRowThreads;
constexpr int row_blocks(int nt, int vpt) {
    const int b = vpt == 4 ? 512 / nt : 2 * kRowThreads / nt;
    return b < 1 ? 1 : b > 8 ? 8 : b;
}
struct RowShape {
    int vpt, nt;
};
RowShape row_shape(int64_t n) {  // for n accesses per row, at most kRowAccesses
    if (n > 4 * 256) return {4, kRowThreads};
    if (n > 2 * kRowThreads) return {4, 256};
    if (n > 2 * 256) return {2, kRowThreads};
    if (n > kRowThreads) return {2, 256};
    for (int nt : {64, 128, 256})
        if (n <= nt) return {1, nt};
    return {1, kRowThreads};
}
#define KDA_ROW_SHAPES(h, X)                             \
    if (h.vpt == 4 && h.nt == 256) { X(4, 256); }        \
    else if (h.vpt == 4) { X(4, kRowThreads); }          \
    else if (h.vpt == 2 && h.nt == 256) { X(2, 256); }   \
    else if (h.vpt == 2) { X(2, kRowThreads); }          \
    else if (h.nt == 64) { X(1, 64); }                   \
    else if (h.nt == 128) { X(1, 128); }                 \
    else if (h.nt == 256) { X(1, 256); }                 \
    else { X(1, kRowThreads); }
// 1 / sqrt(v): the hardware's value r and one Newton step r (1.5 - v r r / 2).  Where v r r is no number (v = 0, or a
// variance that overflowed: r is infinite or 0) r is the result already, the one that 1 / sqrtf(v) has too.
__device__ __forceinline__ float rstd_of(float v) {
    const float r = rsqrtf(v), n = fmaf(-0.5f * (v * r), r, 1.5f);  // v r first: v may be below the normal numbers
    return n == n ? r * n : r;
}

template <typename T, int W, int VPT, int R, int NT>
__global__ void __launch_bounds__(NT, row_blocks(NT, VPT))
k_layer_norm_rows(const T* __restrict__ x, int64_t xs, const float* __restrict__ w, const float* __restrict__ b, float eps,
                  T* __restrict__ y, int64_t ys, float* __restrict__ stats, int64_t M, int C) {
    constexpr int P = W / 2;
    extern __shared__ __align__(16) unsigned char shared[];
    __shared__ __align__(8) float red[2][kMaxWarps][2];
    const float inv_c = 1.0f / (float)C;
    bool in[VPT];  // whether this thread's access i lies inside a row
#pragma unroll
    for (int i = 0; i < VPT; ++i) in[i] = col_of<W, NT>(i) < C;
    f2 wv[VPT][P], bv[VPT][P];
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        const int c = col_of<W, NT>(i);
#pragma unroll
        for (int j = 0; j < P; ++j) {
            wv[i][j] = w && in[i] ? f2_of(w[c + 2 * j], w[c + 2 * j + 1]) : f2_dup(1.f);
            bv[i][j] = b && in[i] ? f2_of(b[c + 2 * j], b[c + 2 * j + 1]) : f2_dup(0.f);
        }
    }
    // The ring: kDepth slots of R rows; a thread's access i of row k lies at slot + (k VPT + i) NT.
    constexpr int kSlot = R * VPT * NT;
    Raw<T, W>* const ring = reinterpret_cast<Raw<T, W>*>(shared) + threadIdx.x;
    const int64_t row_step = (int64_t)gridDim.x, step = R * row_step;
    const T* src = x + blockIdx.x * xs + threadIdx.x * W;  // the row that is copied next
    int64_t src_row = blockIdx.x;
    auto row_sum = [&](float (&v)[2], int b) {
        if constexpr (R == 2) {
            block_sum<NT>(v, red[b]);
        } else {
            float one[1] = {v[0]};
            block_sum<NT>(one, reinterpret_cast<float(*)[1]>(red[b]));
            v[0] = one[0];
        }
    };
    int put = 0, get = 0;  // slots
    auto issue = [&]() {
#pragma unroll
        for (int k = 0; k < R; ++k) {
            if (src_row < M)
#pragma unroll
                for (int i = 0; i < VPT; ++i)
                    if (in[i]) cp_async_raw<T, W>(ring + put + (k * VPT + i) * NT, src + i * NT * W);
            src += row_step * xs;
            src_row += row_step;
        }
        cp_commit();
        put = put + kSlot == kDepth * kSlot ? 0 : put + kSlot;
    };
#pragma unroll
    for (int d = 0; d < kDepth - 1; ++d) issue();
    T* dst = y + blockIdx.x * ys + threadIdx.x * W;
    for (int64_t r0 = blockIdx.x; r0 < M; r0 += step) {
        cp_wait<kDepth - 2>();
        // Each of the three passes reads the rows from the ring again: registers for them would halve the blocks.
        float s[2] = {0.f, 0.f}, mean[2];
#pragma unroll
        for (int k = 0; k < R; ++k) {
            f2 t = f2_dup(0.f);
#pragma unroll
            for (int i = 0; i < VPT; ++i)
                if (in[i]) {
                    f2 v[P];
                    unraw2(ring[get + (k * VPT + i) * NT], v);
#pragma unroll
                    for (int j = 0; j < P; ++j) t = add2(t, v[j]);
                }
            s[k] = f2_sum(t);
        }
        issue();
        row_sum(s, 0);
#pragma unroll
        for (int k = 0; k < R; ++k) {
            mean[k] = s[k] * inv_c;
            f2 t = f2_dup(0.f);
#pragma unroll
            for (int i = 0; i < VPT; ++i)
                if (in[i]) {
                    f2 v[P];
                    unraw2(ring[get + (k * VPT + i) * NT], v);
#pragma unroll
                    for (int j = 0; j < P; ++j) {
                        v[j] = add2(v[j], f2_dup(-mean[k]));
                        t = fma2(v[j], v[j], t);
                    }
                }
            s[k] = f2_sum(t);
        }
        row_sum(s, 1);
#pragma unroll
        for (int k = 0; k < R; ++k) {
            const int64_t r = r0 + k * row_step;
            if (r >= M) break;
            const float rstd = rstd_of(fmaf(s[k], inv_c, eps));
            if (stats && threadIdx.x == 0) *reinterpret_cast<float2*>(stats + 2 * r) = make_float2(mean[k], rstd);
#pragma unroll
            for (int i = 0; i < VPT; ++i) {
                if (!in[i]) continue;
                f2 v[P];
                unraw2(ring[get + (k * VPT + i) * NT], v);
                float o[W];
#pragma unroll
                for (int j = 0; j < P; ++j) {
                    const f2 n = fma2(mul2(add2(v[j], f2_dup(-mean[k])), f2_dup(rstd)), wv[i][j], bv[i][j]);
                    o[2 * j] = f2_lo(n);
                    o[2 * j + 1] = f2_hi(n);
                }
                store_row(dst + i * NT * W, o);
            }
            dst += row_step * ys;
        }
        get = get + kSlot == kDepth * kSlot ? 0 : get + kSlot;
    }
}

template <typename T, bool X8, int W, int VPT>
__global__ void __launch_bounds__(1024)
k_layer_norm_bwd(const T* __restrict__ dy, int64_t dys, const void* __restrict__ xv, int64_t xs,
                 const uint8_t* __restrict__ scales, const float* __restrict__ stats, const float* __restrict__ w,
                 T* __restrict__ dx, int64_t dxs, float* __restrict__ part, int64_t M, int C) {
    using XT = typename std::conditional<X8, uint8_t, T>::type;
    const XT* x = static_cast<const XT*>(xv);
    const int nb = (C + KDA_PACK8_BLOCK - 1) / KDA_PACK8_BLOCK;
    __shared__ __align__(8) float red[2][kMaxWarps][2];
    const float inv_c = 1.0f / (float)C;
    float wv[VPT][W], dw[VPT][W], db[VPT][W];
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        const int c = col_of<W>(i);
#pragma unroll
        for (int j = 0; j < W; ++j) dw[i][j] = db[i][j] = 0.f;
        if (w && c < C) {
            load_param(w + c, wv[i]);
        } else {
#pragma unroll
            for (int j = 0; j < W; ++j) wv[i][j] = 1.f;
        }
    }
    Raw<XT, W> xr[VPT];
    Raw<T, W> yr[VPT];
    uint32_t sr[VPT];
    float mean = 0.f, rstd = 0.f;
    auto fetch = [&](int64_t r) {
        mean = __ldg(stats + 2 * r);
        rstd = __ldg(stats + 2 * r + 1);
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int c = col_of<W>(i);
            if (c < C) {
                xr[i].load(x + r * (X8 ? (int64_t)C : xs) + c);
                yr[i].load(dy + r * dys + c);
                sr[i] = X8 ? (uint32_t)__ldg(scales + r * nb + c / KDA_PACK8_BLOCK) : 0u;
            }
        }
    };
    int buf = 0;
    if (blockIdx.x < M) fetch(blockIdx.x);
    for (int64_t r = blockIdx.x; r < M; r += gridDim.x) {
        float xh[VPT][W], p[VPT][W], s[2] = {0.f, 0.f};
        const float rs = rstd;
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            if (col_of<W>(i) >= C) continue;
            if constexpr (X8) unraw8(xr[i], scale_of_byte(sr[i]), xh[i]); else unraw(xr[i], xh[i]);
            unraw(yr[i], p[i]);
#pragma unroll
            for (int j = 0; j < W; ++j) {
                xh[i][j] = (xh[i][j] - mean) * rs;
                dw[i][j] = fmaf(p[i][j], xh[i][j], dw[i][j]);
                db[i][j] += p[i][j];
                p[i][j] *= wv[i][j];
                s[0] += p[i][j];
                s[1] = fmaf(p[i][j], xh[i][j], s[1]);
            }
        }
        const int64_t next = r + gridDim.x;
        if (next < M) fetch(next);
        block_sum(s, red[buf]);
        buf ^= 1;
        const float m0 = s[0] * inv_c, m1 = s[1] * inv_c;
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int c = col_of<W>(i);
            if (c >= C) continue;
#pragma unroll
            for (int j = 0; j < W; ++j) p[i][j] = rs * (p[i][j] - m0 - xh[i][j] * m1);
            store_row(dx + r * dxs + c, p[i]);
        }
    }
    if (!part) return;
    float* pw = part + (int64_t)blockIdx.x * 2 * C;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        const int c = col_of<W>(i);
        if (c >= C) continue;
#pragma unroll
        for (int j = 0; j < W; ++j) {
            pw[c + j] = dw[i][j];
            pw[C + c + j] = db[i][j];
        }
    }
}

// The gradient of many rows in 16-byte layouts, as the forward takes them.
template <typename T, bool X8, int W, int VPT, int R, int NT>
__global__ void __launch_bounds__(NT, row_blocks(NT, VPT))
k_layer_norm_bwd_rows(const T* __restrict__ dy, uint32_t dys, const void* __restrict__ xv, uint32_t xs,
                      const uint8_t* __restrict__ scales, const float* __restrict__ stats, const float* __restrict__ w,
                      T* __restrict__ dx, uint32_t dxs, float* __restrict__ part, int M, int C) {
    using XT = typename std::conditional<X8, uint8_t, T>::type;
    constexpr int P = W / 2;
    extern __shared__ __align__(16) unsigned char shared[];
    __shared__ __align__(16) float red[2][kMaxWarps][4];
    const XT* x = static_cast<const XT*>(xv);
    const int nb = (C + KDA_PACK8_BLOCK - 1) / KDA_PACK8_BLOCK;
    const float inv_c = 1.0f / (float)C;
    bool in[VPT];
#pragma unroll
    for (int i = 0; i < VPT; ++i) in[i] = col_of<W, NT>(i) < C;
    f2 wv[VPT][P], dw[VPT][P], db[VPT][P];
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        const int c = col_of<W, NT>(i);
#pragma unroll
        for (int j = 0; j < P; ++j) {
            dw[i][j] = db[i][j] = f2_dup(0.f);
            wv[i][j] = w && in[i] ? f2_of(w[c + 2 * j], w[c + 2 * j + 1]) : f2_dup(1.f);
        }
    }
    // Two rings, of dy and x, laid out as the forward's.
    constexpr int kSlot = R * VPT * NT;
    Raw<T, W>* const ring_y = reinterpret_cast<Raw<T, W>*>(shared) + threadIdx.x;
    Raw<XT, W>* const ring_x = reinterpret_cast<Raw<XT, W>*>(shared + kDepth * kSlot * sizeof(Raw<T, W>)) + threadIdx.x;
    // Rows are counted in 32 bits and strides in bytes below 4 GB: a row's address is one instruction, and no
    // running pointer holds registers.
    const int row_step = gridDim.x, step = R * row_step;
    const XT* tx = x + threadIdx.x * W;
    const T* ty = dy + threadIdx.x * W;
    T* tdx = dx + threadIdx.x * W;
    auto at = [](auto* base, int r, uint32_t bytes) {
        return reinterpret_cast<decltype(base)>(reinterpret_cast<uintptr_t>(base) + (uint64_t)(uint32_t)r * bytes);
    };
    int put = 0, get = 0;  // slots
    auto issue = [&](int r0) {  // rows r0, r0 + gridDim.x, ..
#pragma unroll
        for (int k = 0; k < R; ++k) {
            const int r = r0 + k * row_step;
            if (r < M) {
                const XT* sx = at(tx, r, xs);
                const T* sy = at(ty, r, dys);
#pragma unroll
                for (int i = 0; i < VPT; ++i)
                    if (in[i]) {
                        cp_async_raw<XT, W>(ring_x + put + (k * VPT + i) * NT, sx + i * NT * W);
                        cp_async_raw<T, W>(ring_y + put + (k * VPT + i) * NT, sy + i * NT * W);
                    }
            }
        }
        cp_commit();
        put = put + kSlot == kDepth * kSlot ? 0 : put + kSlot;
    };
    uint32_t sr[R][VPT];
    float2 st[R];
    auto small = [&](int r0) {  // what the next rows need besides: their statistics and their blocks' scales
#pragma unroll
        for (int k = 0; k < R; ++k) {
            const int r = r0 + k * row_step;
            st[k] = make_float2(0.f, 0.f);
#pragma unroll
            for (int i = 0; i < VPT; ++i) sr[k][i] = 127;
            if (r < M) {
                st[k] = __ldg(at(reinterpret_cast<const float2*>(stats), r, 8));
                if (X8)
#pragma unroll
                    for (int i = 0; i < VPT; ++i)
                        if (in[i]) sr[k][i] = (uint32_t)__ldg(at(scales, r, nb) + col_of<W, NT>(i) / KDA_PACK8_BLOCK);
            }
        }
    };
#pragma unroll
    for (int d = 0; d < kDepth - 1; ++d) issue(blockIdx.x + d * step);
    small(blockIdx.x);
    int buf = 0;
    for (int r0 = blockIdx.x; r0 < M; r0 += step) {
        cp_wait<kDepth - 2>();
        float rs[R], mean[R];
        uint32_t sc[R][VPT];
        float s[4] = {0.f, 0.f, 0.f, 0.f};
        // x - mean and dy of one access, from the ring: read once for the sums and once for dx, since registers for
        // them would halve the blocks.  The mean is subtracted from x itself (x rstd - mean rstd in one multiply-add
        // would round at the size of mean / deviation), and rstd comes to the sums and factors where that is free.
        auto terms = [&](int k, int i, f2 (&xm)[P], f2 (&d)[P]) {
            unraw2(ring_x[get + (k * VPT + i) * NT], xm);
            unraw2(ring_y[get + (k * VPT + i) * NT], d);
            const f2 m = f2_dup(-mean[k]), scale = f2_dup(scale_of_byte(sc[k][i]));
#pragma unroll
            for (int j = 0; j < P; ++j) xm[j] = X8 ? fma2(xm[j], scale, m) : add2(xm[j], m);
        };
#pragma unroll
        for (int k = 0; k < R; ++k) {
            rs[k] = st[k].y;
            mean[k] = st[k].x;
#pragma unroll
            for (int i = 0; i < VPT; ++i) sc[k][i] = sr[k][i];
            if (R > 1 && r0 + k * row_step >= M) continue;  // its slot holds no row
            f2 a = f2_dup(0.f), b = f2_dup(0.f);
#pragma unroll
            for (int i = 0; i < VPT; ++i) {
                if (!in[i]) continue;
                f2 xm[P], d[P];
                terms(k, i, xm, d);
#pragma unroll
                for (int j = 0; j < P; ++j) {
                    const f2 xh = mul2(xm[j], f2_dup(rs[k]));
                    dw[i][j] = fma2(d[j], xh, dw[i][j]);
                    db[i][j] = add2(db[i][j], d[j]);
                    d[j] = mul2(d[j], wv[i][j]);
                    a = add2(a, d[j]);
                    b = fma2(d[j], xh, b);
                }
            }
            s[2 * k] = f2_sum(a);
            s[2 * k + 1] = f2_sum(b);
        }
        issue(r0 + (kDepth - 1) * step);
        small(r0 + step);
        if constexpr (R == 1) {
            float t[2] = {s[0], s[1]};
            block_sum<NT>(t, reinterpret_cast<float(*)[2]>(red[buf]));
            s[0] = t[0];
            s[1] = t[1];
        } else {
            block_sum4<NT>(s, red[buf]);
        }
        buf ^= 1;
#pragma unroll
        for (int k = 0; k < R; ++k) {
            if (R > 1 && r0 + k * row_step >= M) break;
            const f2 m0 = f2_dup(-s[2 * k] * inv_c), m1 = f2_dup(-s[2 * k + 1] * inv_c * rs[k]), rr = f2_dup(rs[k]);
#pragma unroll
            for (int i = 0; i < VPT; ++i) {
                if (!in[i]) continue;
                f2 xm[P], d[P];
                terms(k, i, xm, d);
                float o[W];
#pragma unroll
                for (int j = 0; j < P; ++j) {
                    const f2 v = mul2(rr, fma2(xm[j], m1, fma2(d[j], wv[i][j], m0)));
                    o[2 * j] = f2_lo(v);
                    o[2 * j + 1] = f2_hi(v);
                }
                store_row(at(tdx, r0 + k * row_step, dxs) + i * NT * W, o);
            }
        }
        get = get + kSlot == kDepth * kSlot ? 0 : get + kSlot;
    }
    if (!part) return;
    float* pw = part + (int64_t)blockIdx.x * 2 * C;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        const int c = col_of<W, NT>(i);
        if (c >= C) continue;
#pragma unroll
        for (int j = 0; j < P; ++j) {
            *reinterpret_cast<float2*>(pw + c + 2 * j) = make_float2(f2_lo(dw[i][j]), f2_hi(dw[i][j]));
            *reinterpret_cast<float2*>(pw + C + c + 2 * j) = make_float2(f2_lo(db[i][j]), f2_hi(db[i][j]));
        }
    }
}

struct PutParams {  // column c of [dw | db]
    float *dw, *db;
    int C;
    __device__ void operator()(int64_t c, float s) const {
        if (c < C) {
            if (dw) dw[c] = s;
        } else if (db) {
            db[c - C] = s;
        }
    }
};

bool vec_ok(const void* p, int64_t stride, int esize, int w) {
    return reinterpret_cast<uintptr_t>(p) % (w * esize) == 0 && stride % w == 0;
}
bool par_ok(const float* p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; }
int warps32(int64_t n) { return (int)((n + 31) / 32 * 32); }

// Accesses per thread: the fewest of {1, 2, 4, 8, last} that keep a row within `most` threads.
int accesses(int64_t n, int most, int last) {
    for (int v : {1, 2, 4, 8})
        if (n <= (int64_t)v * most) return v;
    return last;
}

}  // namespace

cudaError_t launch_layer_norm(const kda_norm_args& a, cudaStream_t s) {
    const int es = a.io == KDA_BF16 ? 2 : 4, vw = 16 / es;
    const int64_t xs = a.x_stride ? a.x_stride : a.C, ys = a.y_stride ? a.y_stride : a.C;
    const bool vec = a.C % vw == 0 && vec_ok(a.x, xs, es, vw) && vec_ok(a.y, ys, es, vw) &&
                     par_ok(a.weight) && par_ok(a.bias);
    const int64_t n = vec ? a.C / vw : a.C;
    DeviceInfo di{0, 0, 0};
    const int sms = current_device_info(&di) ? di.sm_count : 1;
    // Single elements: the more rows there are, the fewer threads take one, with more loads in flight each and fewer
    // warps at a barrier (20,000 x 333 bf16: 22 us with at most 64 threads, 24 with 128, 47 with 512; 1,237 x 1,001 fp32:
    // 9.6, 6.4 and 8.2; 300 x 1,001: 9.0, 3.8 and 2.8).
    const int most = vec || a.M < 4 * (int64_t)sms ? 512 : a.M < 16 * (int64_t)sms ? 128 : 64;
    const int vpt = accesses(n, most, vec ? 16 : 32);
    const int nt = warps32((n + vpt - 1) / vpt);
    // Rows through shared memory once every SM has several of them to take in turn (the ring needs rows to
    // come): 8,192 x 7,168 bf16.  Fewer rows go one per block.
    if (vec && n <= kRowAccesses) {
        const RowShape h = row_shape(n);
        const int smem = kDepth * (h.vpt == 4 ? 1 : 2) * h.vpt * h.nt * 16, per_sm = row_blocks(h.nt, h.vpt);
        if (a.M >= 4 * (int64_t)sms * per_sm) {
            cudaError_t e = cudaSuccess;
#define KDA_LNR(T, W, V, NT)                                                                                         \
    if (!(e = cudaFuncSetAttribute(k_layer_norm_rows<T, W, V, V == 4 ? 1 : 2, NT>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem))) \
        k_layer_norm_rows<T, W, V, V == 4 ? 1 : 2, NT><<<sms * per_sm, NT, smem, s>>>(                                            \
            static_cast<const T*>(a.x), xs, a.weight, a.bias, a.eps, static_cast<T*>(a.y), ys, a.stats, a.M, a.C)
#define KDA_LNR_B(V, NT) KDA_LNR(bf16, 8, V, NT)
#define KDA_LNR_F(V, NT) KDA_LNR(float, 4, V, NT)
            if (a.io == KDA_BF16) { KDA_ROW_SHAPES(h, KDA_LNR_B) } else { KDA_ROW_SHAPES(h, KDA_LNR_F) }
#undef KDA_LNR_F
#undef KDA_LNR_B
#undef KDA_LNR
            return e ? e : cudaGetLastError();
        }
    }
    const unsigned grid = (unsigned)(a.M < 0x7fffffff ? a.M : 0x7fffffff);
#define KDA_LN(T, W, V)                                                                                       \
    k_layer_norm<T, W, V><<<grid, nt, 0, s>>>(static_cast<const T*>(a.x), xs, a.weight, a.bias, a.eps,         \
                                              static_cast<T*>(a.y), ys, a.stats, a.M, a.C)
#define KDA_LN_V(T, W)                                                                                        \
    switch (vpt) {                                                                                            \
        case 1: KDA_LN(T, W, 1); break;                                                                       \
        case 2: KDA_LN(T, W, 2); break;                                                                       \
        case 4: KDA_LN(T, W, 4); break;                                                                       \
        case 8: KDA_LN(T, W, 8); break;                                                                       \
        default: KDA_LN(T, W, (W == 1 ? 32 : W == 4 ? 16 : 8)); break; /* bf16 vectors never need more than 8 */ \
    }
    if (a.io == KDA_BF16) {
        if (vec) { KDA_LN_V(bf16, 8) } else { KDA_LN_V(bf16, 1) }
    } else {
        if (vec) { KDA_LN_V(float, 4) } else { KDA_LN_V(float, 1) }
    }
#undef KDA_LN_V
#undef KDA_LN
    return cudaGetLastError();
}

namespace {
struct BwdShape {
    bool vec;
    int vpt, nt;
};
BwdShape bwd_shape(const kda_norm_backward_args& a) {
    const int es = a.io == KDA_BF16 ? 2 : 4, vw = 16 / es;
    const int64_t dys = a.dy_stride ? a.dy_stride : a.C, dxs = a.dx_stride ? a.dx_stride : a.C;
    const int64_t xs = a.x_stride ? a.x_stride : a.C;
    BwdShape h;
    h.vec = a.C % vw == 0 && vec_ok(a.dy, dys, es, vw) && vec_ok(a.dx, dxs, es, vw) && par_ok(a.weight) &&
            (a.x_scales ? vec_ok(a.x, a.C, 1, vw) : vec_ok(a.x, xs, es, vw));
    const int64_t n = h.vec ? a.C / vw : a.C;
    // Single elements: up to eight per thread, for the same reasons as in the forward pass (1,237 x 1,001 fp32: 5.4 us
    // against 7.4 with one), more only where a row needs them.
    h.vpt = accesses(n, h.vec || n > 8 * 256 ? 1024 : 256, 32);
    h.nt = warps32((n + h.vpt - 1) / h.vpt);
    return h;
}
}  // namespace

NormBackwardPlan norm_backward_plan(const kda_norm_backward_args& a) {
    NormBackwardPlan p{0, 0};
    DeviceInfo di{0, 0, 0};
    const int sms = current_device_info(&di) ? di.sm_count : 1;
    // Blocks that fill an SM's threads when the layout allows 16-byte accesses (known only once the
    // pointers are; the sizes alone have to fix the workspace).
    const int vw = a.io == KDA_BF16 ? 8 : 4, acc = (a.C + vw - 1) / vw;
    const RowShape h = acc <= kRowAccesses ? row_shape(acc) : RowShape{4, kRowThreads};
    const int per_sm = row_blocks(h.nt, h.vpt);
    const int64_t most = (int64_t)sms * per_sm;
    p.blocks = (int)(a.M < most ? a.M : most);
    p.workspace = (a.dweight || a.dbias) ? (size_t)p.blocks * 2 * a.C * sizeof(float) : 0;
    return p;
}

cudaError_t launch_layer_norm_backward(const kda_norm_backward_args& a, const NormBackwardPlan& p, cudaStream_t s) {
    const BwdShape h = bwd_shape(a);
    const int64_t dys = a.dy_stride ? a.dy_stride : a.C, dxs = a.dx_stride ? a.dx_stride : a.C;
    const int64_t xs = a.x_stride ? a.x_stride : a.C;
    float* part = p.workspace ? static_cast<float*>(a.workspace) : nullptr;
    cudaError_t e = cudaSuccess;
    const int es = a.io == KDA_BF16 ? 2 : 4;
    const int acc = a.C / (16 / es);  // accesses per row, where the layout is wide
    const int64_t most = (int64_t)0xffffffff / es;  // elements of a row stride below 4 GB
    if (h.vec && acc <= kRowAccesses && a.M < (1 << 30) && dys <= most && dxs <= most && xs <= most) {
        const RowShape r = row_shape(acc);
        const int smem = kDepth * (r.vpt == 1 ? 2 : 1) * r.vpt * r.nt * (16 + (a.x_scales ? 16 / es : 16));
#define KDA_LNBR(T, X8, W, V, NT)                                                                                    \
    if (!(e = cudaFuncSetAttribute(k_layer_norm_bwd_rows<T, X8, W, V, V == 1 ? 2 : 1, NT>,                                    \
                                   cudaFuncAttributeMaxDynamicSharedMemorySize, smem)))                              \
        k_layer_norm_bwd_rows<T, X8, W, V, V == 1 ? 2 : 1, NT><<<p.blocks, NT, smem, s>>>(                                    \
            static_cast<const T*>(a.dy), (uint32_t)(dys * es), a.x, (uint32_t)(a.x_scales ? a.C : xs * es), a.x_scales, \
            a.stats, a.weight, static_cast<T*>(a.dx), (uint32_t)(dxs * es), part, (int)a.M, a.C)
#define KDA_LNBR_B8(V, NT) KDA_LNBR(bf16, true, 8, V, NT)
#define KDA_LNBR_B(V, NT) KDA_LNBR(bf16, false, 8, V, NT)
#define KDA_LNBR_F8(V, NT) KDA_LNBR(float, true, 4, V, NT)
#define KDA_LNBR_F(V, NT) KDA_LNBR(float, false, 4, V, NT)
        if (a.io == KDA_BF16) {
            if (a.x_scales) { KDA_ROW_SHAPES(r, KDA_LNBR_B8) } else { KDA_ROW_SHAPES(r, KDA_LNBR_B) }
        } else {
            if (a.x_scales) { KDA_ROW_SHAPES(r, KDA_LNBR_F8) } else { KDA_ROW_SHAPES(r, KDA_LNBR_F) }
        }
#undef KDA_LNBR_F
#undef KDA_LNBR_F8
#undef KDA_LNBR_B
#undef KDA_LNBR_B8
#undef KDA_LNBR
        if (!e) e = cudaGetLastError();
        if (e || !part) return e;
        return launch_column_sum(part, p.blocks, 2 * (int64_t)a.C, PutParams{a.dweight, a.dbias, a.C}, s);
    }
#define KDA_LNB(T, X8, W, V)                                                                                   \
    k_layer_norm_bwd<T, X8, W, V><<<p.blocks, h.nt, 0, s>>>(static_cast<const T*>(a.dy), dys, a.x, xs,          \
                                                            a.x_scales, a.stats, a.weight,                      \
                                                            static_cast<T*>(a.dx), dxs, part, a.M, a.C)
#define KDA_LNB_V(T, X8, W)                                                                                    \
    switch (h.vpt) {                                                                                           \
        case 1: KDA_LNB(T, X8, W, 1); break;                                                                   \
        case 2: KDA_LNB(T, X8, W, 2); break;                                                                   \
        case 4: KDA_LNB(T, X8, W, 4); break;                                                                   \
        case 8: KDA_LNB(T, X8, W, (W == 8 ? 4 : 8)); break;                                                    \
        default: KDA_LNB(T, X8, W, (W == 1 ? 32 : W == 4 ? 8 : 4)); break; /* vectors: never more than these */ \
    }
#define KDA_LNB_X(T, W)                                                                                        \
    if (a.x_scales) { KDA_LNB_V(T, true, W) } else { KDA_LNB_V(T, false, W) }
    if (a.io == KDA_BF16) {
        if (h.vec) { KDA_LNB_X(bf16, 8) } else { KDA_LNB_X(bf16, 1) }
    } else {
        if (h.vec) { KDA_LNB_X(float, 4) } else { KDA_LNB_X(float, 1) }
    }
#undef KDA_LNB_X
#undef KDA_LNB_V
#undef KDA_LNB
    e = cudaGetLastError();
    if (e || !part) return e;
    return launch_column_sum(part, p.blocks, 2 * (int64_t)a.C, PutParams{a.dweight, a.dbias, a.C}, s);
}

}  // namespace kda
