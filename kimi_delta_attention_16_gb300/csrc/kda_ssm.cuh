// kda_ssm.cuh -- what the selective scan's kernels share: the step size, the thread layout over
// (channel, state) and the walk over packed sequences.
#pragma once

#include "kda_block.cuh"

namespace kda {
namespace ssm {

// softplus(x) = max(x, 0) + log(1 + e^-|x|), to a few units of the last place for every x: the
// logarithm as 2 atanh(s), s = e / (2 + e) <= 1/3, by its odd power series up to s^13 (the next
// term is below 2^-26 of the sum).  log(1 + e) directly would lose the digits of a small e.
__device__ __forceinline__ float softplus(float x) {
    const float e = expf(-fabsf(x));
    const float s = __fdividef(e, 2.f + e), q = s * s;
    float p = 1.f / 13.f;
    p = fmaf(p, q, 1.f / 11.f);
    p = fmaf(p, q, 1.f / 9.f);
    p = fmaf(p, q, 1.f / 7.f);
    p = fmaf(p, q, 1.f / 5.f);
    p = fmaf(p, q, 1.f / 3.f);
    p = fmaf(p, q, 1.f);
    return fmaxf(x, 0.f) + 2.f * s * p;
}
__device__ __forceinline__ float sigmoid(float x) { return __fdividef(1.f, 1.f + expf(-x)); }
__device__ __forceinline__ float silu(float x) { return __fdividef(x, 1.f + expf(-x)); }

// 2^x of both halves.
__device__ __forceinline__ f2 exp2_2(f2 x) { return f2_of(exp2_hw(f2_lo(x)), exp2_hw(f2_hi(x))); }

template <typename T> __device__ __forceinline__ float ldf(const T* p) {
    Raw<T, 1> r;
    r.load(p);
    float v[1];
    unraw(r, v);
    return v[0];
}

// One call's arguments as the kernels take them (strides in elements, never 0).
struct Params {
    const void *u, *dt, *z, *B, *Cm;
    void* y;
    int64_t us, dts, zs, bs, cs, ys;
    const float *A, *D, *dt_bias, *init;
    float* fin;
    const int32_t* cu;
    float *ws_state, *ws_sum;
    int64_t T, piece;
    int N, C, G, Cg, bpg;  // sequences, channels, groups, channels and blocks per group
    int pieces, softplus;
};

constexpr int kCB = 64;  // channels per block

// Block of kCB channels (32 pairs c, c + 32) x NS states: a thread holds 4 states of both channels
// of a pair.  The lanes of a warp that share states are neighbours, so a token's B and C, four
// floats per lane, take two shared-memory cycles per warp instead of four.
template <int NS> struct Lay {
    static constexpr int L = NS / 4;          // threads along the states
    static constexpr int kThreads = 32 * L;
    static constexpr int KPW = 32 / L;        // channel pairs per warp
    static constexpr int TT = NS == 64 ? 8 : 16;  // tokens per tile
    static constexpr int EPT = TT * kCB / kThreads;  // (token, channel) elements per thread and tile
    static constexpr int BPT = TT * NS / kThreads;   // elements of B (and C) per thread and tile
};

}  // namespace ssm
}  // namespace kda
