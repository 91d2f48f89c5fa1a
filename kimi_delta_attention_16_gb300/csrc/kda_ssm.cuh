// kda_ssm.cuh -- what the selective scan's kernels share: the step size, the thread layout over
// (channel, state) and the walk over packed sequences.
#pragma once

#include "kda_block.cuh"

namespace kda {
namespace ssm {

// The larger of two values, NaN where one is NaN.
__device__ __forceinline__ float max_nan(float a, float b) {
    float m;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(m) : "f"(a), "f"(b));
    return m;
}
constexpr float kLn2 = 0.6931471805599453f;

// softplus(x) = max(x, 0) + log(1 + e^-|x|), to a dozen units of 2^-24 (four of them the hardware exponential's).
// e^-|x| = 2^h (1 + r) with h = -|x| log2 e as rounded and r = -|x| - h ln 2 what that left out (one multiply-add: the
// product is exact); without r the exponent's rounding would cost |x| units more, 10 where trained step sizes lie.
// From -104 on e^-|x| is 0 in fp32; the bound keeps h finite.  The
// logarithm as 2 atanh(s) = s P(s^2), s = e / (2 + e) <= 1/3, with a polynomial of degree 4 fitted to the quotient
// 2 atanh(s) / s over s^2 in [0, 1/9] (relative error 2^-26; its power series would take degree 6).
// log(1 + e) directly would lose the digits of a small e.  Both halves of a pair at once.
__device__ __forceinline__ f2 softplus2(f2 x) {
    const f2 t = f2_of(max_nan(-fabsf(f2_lo(x)), -104.f), max_nan(-fabsf(f2_hi(x)), -104.f));
    const f2 h = mul2(t, f2_dup(kLog2e)), r = fma2(h, f2_dup(-kLn2), t);
    const f2 e0 = f2_of(exp2_hw(f2_lo(h)), exp2_hw(f2_hi(h))), e = fma2(e0, r, e0);
    const f2 d = add2(e, f2_dup(2.f));
    const f2 s = mul2(e, f2_of(rcp_hw(f2_lo(d)), rcp_hw(f2_hi(d)))), q = mul2(s, s);
    f2 p = f2_dup(0.2817833423614502f);
    p = fma2(p, q, f2_dup(0.27960604429244995f));
    p = fma2(p, q, f2_dup(0.40024909377098083f));
    p = fma2(p, q, f2_dup(0.6666631698608398f));
    p = fma2(p, q, f2_dup(2.f));
    return fma2(s, p, f2_of(fmaxf(f2_lo(x), 0.f), fmaxf(f2_hi(x), 0.f)));
}
__device__ __forceinline__ float softplus(float x) { return f2_lo(softplus2(f2_of(x, 0.f))); }

// One call's arguments as the kernels take them (strides in elements, never 0).
struct Params {
    const void *u, *dt, *z, *B, *Cm;
    void* y;
    int64_t us, dts, zs, bs, cs, ys;
    const float *A, *D, *dt_bias, *init;
    float* fin;
    const int32_t* cu;
    float *ws_state, *ws_sum, *ckpt;
    int64_t T, piece;
    int N, C, G, Cg;  // sequences, channels, groups, channels per group
    int pieces, softplus;
    bool vec;   // 16-byte copies of every row, strides below 4 GB
    bool wide;  // two channels per access to y
};

Params params_of(const kda_ssm_args& a);  // everything but the pieces and the workspace
// The state in front of every fourth token to p.ckpt [ceil(T / 4)][C][NS] (pieces start at multiples of 8).
cudaError_t launch_states(const Params& p, const kda_ssm_args& a, cudaStream_t s);

// Two neighbouring elements (aligned to both).
__device__ __forceinline__ f2 pair_of(const float* v) {
    const float2 f = *reinterpret_cast<const float2*>(v);
    return f2_of(f.x, f.y);
}
__device__ __forceinline__ f2 pair_of(const bf16* v) {
    const uint32_t w = *reinterpret_cast<const uint32_t*>(v);
    return f2_of(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}
__device__ __forceinline__ void put2(float* o, f2 v) { *reinterpret_cast<float2*>(o) = make_float2(f2_lo(v), f2_hi(v)); }
__device__ __forceinline__ void put2(bf16* o, f2 v) {
    *reinterpret_cast<__nv_bfloat162*>(o) = __floats2bfloat162_rn(f2_lo(v), f2_hi(v));
}

// Block of CB channels x NS states: a thread holds up to 16 states of CPT neighbouring channels, L threads
// share them.  Lanes that hold the same states are neighbours, so they read a token's B and C at one
// shared-memory address (broadcast).
template <int NS, int kChannels> struct Lay {
    static constexpr int CPT = kChannels;
    static constexpr int SPT = NS < 16 ? NS : 16;  // states per thread and channel
    static constexpr int L = NS / SPT;             // threads per channel
    static constexpr int NT = 64;                  // threads per block
    static constexpr int CB = CPT * NT / L;        // channels per block
    static constexpr int KPW = 32 / L;             // threads along the channels per warp
    static constexpr int TT = 8;                   // tokens per tile
    static constexpr int BPT = TT * NS / NT;       // elements of B (and C) per thread and tile
    static_assert(BPT >= 1, "tile too small");
};

// ------------------------------------------------------------------ joining the pieces
constexpr int kJoinThreads = 128;
constexpr int kMaxPieces = 1024;  // of a plan
constexpr int kJoinBits = kMaxPieces;

// Bit k: nothing passes through piece k.  From the left (kDir = 1) because a sequence starts in it, at its first
// token or inside; from the right (kDir = -1) because one ends in it, inside or at its last token.  The two differ where
// a sequence's border is a piece's: its end closes the piece before, its start the piece behind.
template <int kDir> __device__ __forceinline__ void mark_closed(const Params& p, uint32_t (&bits)[kJoinBits / 32]) {
    for (int k = threadIdx.x; k < kJoinBits; k += kJoinThreads) {
        bool s = false;
        if (k < p.pieces) {
            const int64_t t0 = k * p.piece, t1 = t0 + p.piece < p.T ? t0 + p.piece : p.T;
            s = kDir > 0 ? p.cu[seq_of(p.cu, p.N, t1 - 1)] >= t0 : p.cu[seq_of(p.cu, p.N, t0) + 1] <= t1;
        }
        const uint32_t w = __ballot_sync(0xffffffffu, s);
        if ((threadIdx.x & 31) == 0) bits[k / 32] = w;
    }
    __syncthreads();
}

// carry = (carry, unless the piece is closed to it) 2^(a2 sum of delta) + the piece's own, over
// `count` pieces from `k` on (kDir: +1 or -1), each result written over the own one.  Eight pieces' values
// are loaded before the first is used: the chain is one multiply-add per piece, not one latency.
template <int kDir>
__device__ __forceinline__ void join(const Params& p, const uint32_t* closed, int k, int count, float a2, float carry,
                                     float* slot, const float* sum, int64_t row) {
    constexpr int U = 8;
    for (int c = 0; c < count; c += U) {
        float o[U], f[U];
#pragma unroll
        for (int j = 0; j < U; ++j) {
            const int64_t q = k + (int64_t)kDir * (c + j);
            o[j] = c + j < count ? slot[q * row] : 0.f;
            f[j] = c + j < count ? sum[q * p.C] : 0.f;
        }
#pragma unroll
        for (int j = 0; j < U; ++j) {
            if (c + j >= count) break;
            const int64_t q = k + (int64_t)kDir * (c + j);
            carry = closed[q / 32] >> (q & 31) & 1 ? o[j] : fmaf(exp2_hw(a2 * f[j]), carry, o[j]);
            slot[q * row] = carry;
        }
    }
}

// ------------------------------------------------------------------ tiles of rows through shared memory
// Rows [row, row + rows) of a tensor (W columns from `first`, of which `cols` exist) to dst[TT][W]: asynchronous
// 16-byte copies where the layout allows them, plain element copies otherwise.  What does not exist is not written.
// A thread's pieces are the same columns of every tile, so a copy is a row's address (32 x 32 bits to 64, one
// instruction: `vec` stands for row strides below 4 GB too) and the copy itself (8,192 tokens x 12,288 channels x 16:
// 770 -> 730 us against 64-bit index arithmetic and partial pieces).
template <typename T, int TT, int W, int NT>
__device__ __forceinline__ void copy_tile(T* dst, const T* first, int64_t stride, uint32_t row, int rows, int cols, bool vec) {
    if (vec) {
        constexpr int E = 16 / (int)sizeof(T), PR = W / E, N = TT * PR;  // elements per piece, pieces per row and tile
        static_assert(W % E == 0 && NT % PR == 0, "a thread keeps its columns");
        const int c = (int)threadIdx.x % PR * E, r = (int)threadIdx.x / PR;
        const char* col = reinterpret_cast<const char*>(first + c);
        const uint32_t bytes = (uint32_t)stride * (uint32_t)sizeof(T);
        if (c < cols)
#pragma unroll
            for (int k = 0; k < (N + NT - 1) / NT; ++k) {
                const int rk = r + k * (NT / PR);
                if (rk < rows)
                    cp_async16(dst + (k * NT + (int)threadIdx.x) * E, col + (uint64_t)(row + rk) * bytes);
            }
    } else {
#pragma unroll 4
        for (int i = threadIdx.x; i < TT * W; i += NT) {
            const int r = i / W, c = i % W;
            if (r < rows && c < cols) dst[i] = first[(int64_t)(row + r) * stride + c];
        }
    }
}

}  // namespace ssm
}  // namespace kda
