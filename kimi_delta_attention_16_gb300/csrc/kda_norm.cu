// kda_norm.cu -- layer norm over the last axis, forward and backward.
//
//   forward   mean, var = mean of squared deviations, y = (x - mean) rstd w + b
//   backward  xh = (x - mean) rstd, p = dy w:
//             dx = rstd (p - mean(p) - xh mean(p xh)),  dw = sum_rows dy xh,  db = sum_rows dy
//
// Both are bound by HBM: one read of x (and dy), one write of y (dx).  A row lives in the
// registers of one block (VPT accesses of W elements per thread), so the statistics take two
// passes over registers, none over memory.  The backward is persistent: a thread owns the same
// columns in every row of its block, keeps their dw and db sums in registers and leaves one
// partial per block, which k_column_sum adds up in block order (no atomics: the same bits
// every time).  The next row's accesses are issued before the current row's sums.
#include "kda_block.cuh"

namespace kda {

namespace {

constexpr int kMaxWarps = 32;

// Sum over the block; every thread gets it.  `buf` is written and read once: a caller that comes
// back to the same buffer has passed another barrier in between.
template <int K> __device__ __forceinline__ void block_sum(float (&v)[K], float (*buf)[K]) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) v[k] += __shfl_xor_sync(0xffffffffu, v[k], o);
    if (nw == 1) return;
    if (lane == 0)
#pragma unroll
        for (int k = 0; k < K; ++k) buf[warp][k] = v[k];
    __syncthreads();
#pragma unroll
    for (int k = 0; k < K; ++k) {
        v[k] = lane < nw ? buf[lane][k] : 0.f;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) v[k] += __shfl_xor_sync(0xffffffffu, v[k], o);
    }
}

// Column of access i of this thread (in elements): consecutive threads take consecutive accesses.
template <int W> __device__ __forceinline__ int col_of(int i) {
    return (i * (int)blockDim.x + (int)threadIdx.x) * W;
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

template <typename T, bool X8, int W, int VPT>
__global__ void __launch_bounds__(1024)
k_layer_norm_bwd(const T* __restrict__ dy, int64_t dys, const void* __restrict__ xv, int64_t xs,
                 const uint8_t* __restrict__ scales, const float* __restrict__ stats, const float* __restrict__ w,
                 T* __restrict__ dx, int64_t dxs, float* __restrict__ part, int64_t M, int C) {
    using XT = typename std::conditional<X8, uint8_t, T>::type;
    const XT* x = static_cast<const XT*>(xv);
    const int nb = (C + KDA_PACK8_BLOCK - 1) / KDA_PACK8_BLOCK;
    __shared__ float red[2][kMaxWarps][2];
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
    const int vpt = accesses(n, 512, vec ? 16 : 32);
    const int nt = warps32((n + vpt - 1) / vpt);
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
        default: KDA_LN(T, W, (W == 1 ? 32 : 16)); break;                                                     \
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
    h.vpt = accesses(n, 1024, 32);
    h.nt = warps32((n + h.vpt - 1) / h.vpt);
    return h;
}
}  // namespace

NormBackwardPlan norm_backward_plan(const kda_norm_backward_args& a) {
    NormBackwardPlan p{0, 0};
    DeviceInfo di{0, 0, 0};
    const int sms = current_device_info(&di) ? di.sm_count : 1;
    const int nt = warps32(a.C < 1024 ? a.C : 1024);  // an upper bound on the threads of any layout
    int per_sm = 1024 / nt;
    if (per_sm > 8) per_sm = 8;
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
#define KDA_LNB(T, X8, W, V)                                                                                   \
    k_layer_norm_bwd<T, X8, W, V><<<p.blocks, h.nt, 0, s>>>(static_cast<const T*>(a.dy), dys, a.x, xs,          \
                                                            a.x_scales, a.stats, a.weight,                      \
                                                            static_cast<T*>(a.dx), dxs, part, a.M, a.C)
#define KDA_LNB_V(T, X8, W)                                                                                    \
    switch (h.vpt) {                                                                                           \
        case 1: KDA_LNB(T, X8, W, 1); break;                                                                   \
        case 2: KDA_LNB(T, X8, W, 2); break;                                                                   \
        case 4: KDA_LNB(T, X8, W, 4); break;                                                                   \
        case 8: KDA_LNB(T, X8, W, 8); break;                                                                   \
        default: KDA_LNB(T, X8, W, (W == 1 ? 32 : 8)); break; /* vectors never need more than 8 */                                                  \
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
    cudaError_t e = cudaGetLastError();
    if (e || !part) return e;
    return launch_column_sum(part, p.blocks, 2 * (int64_t)a.C, PutParams{a.dweight, a.dbias, a.C}, s);
}

}  // namespace kda
