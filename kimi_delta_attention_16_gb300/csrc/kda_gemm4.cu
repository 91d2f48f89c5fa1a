// kda_gemm4.cu -- C[M][N] = epilogue(A[M][K] . W[N][K]^T) for few rows of A and weights in 4 bits
// (e2m1 or offset integers under one scale per group): the projections of a decode step.
//
// What a call has to read is N K / 2 bytes of codes and their scales.  e2m1 weights go through the block-scaled tensor
// cores (kda_few_tc.cuh), integer codes through registers (kda_few.cuh).  A CTA takes 128 of the N outputs for some
// tokens, a cluster splits K.
#include "kda_few.cuh"
#include "kda_few_tc.cuh"
#include "kda_serve.cuh"

namespace kda {

namespace {

using namespace few;

struct Gemm4 {
    Matrix w;
    int M, N, K, epi, ranks;
    const bf16* a;
    int64_t lda;
    bool wide;
    int64_t ldc;
};

template <int F, int NT, typename Tout>
__global__ void __launch_bounds__(kThreads, 2) k_gemm4(const Gemm4 p, Tout* __restrict__ out) {
    using L = Layout<F, NT>;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ int of[L::cols];
    const int rank = blockIdx.x % p.ranks, row0 = blockIdx.x / p.ranks * kTileRows;
    const int c0 = blockIdx.y * L::cols, n = min(L::cols, p.M - c0);
    if (threadIdx.x < L::cols) of[threadIdx.x] = c0 + threadIdx.x;
    __syncthreads();
    int k0, k1;
    slice_of(p.K, rank, p.ranks, k0, k1);
    const auto row_of = [&](int r) { return (int64_t)min(row0 + r, p.N - 1); };
    float acc[NT][4];
    product<F, NT>(smem, p.w, p.K, row_of, Bf16Rows{p.a, p.lda, p.wide}, of, n, k0, k1, acc);
    float* red = gather<F, NT>(smem, acc, p.ranks);
    const int share = kTileRows / p.ranks;
    for (int i = threadIdx.x; i < n * share; i += kThreads) {
        const int c = i / share, r = rank * share + i % share;
        if (row0 + r >= p.N) continue;
        float v = joined<1>(red, p.ranks, c, r);
        if (p.epi != KDA_EPI_NONE) v = (p.epi == KDA_EPI_DECAY ? -5.0f : 1.0f) / (1.0f + expf(-v));
        out[(int64_t)(c0 + c) * p.ldc + row0 + r] = from_f<Tout>(v);
    }
    if (p.ranks > 1) release(p.ranks);
}

template <int F, int NT, typename Tout> cudaError_t launch(const kda_gemm4_args& a, int ranks, cudaStream_t s) {
    using L = Layout<F, NT>;
    Gemm4 p;
    p.w = Matrix{a.codes, a.scales, a.format == KDA_WEIGHT_E2M1 ? 0 : a.scale_dtype == KDA_BF16 ? 1 : 2, group_shift(a.group)};
    p.M = a.M, p.N = a.N, p.K = a.K, p.epi = a.epilogue, p.ranks = ranks;
    p.a = static_cast<const bf16*>(a.A), p.lda = a.lda;
    p.wide = reinterpret_cast<uintptr_t>(a.A) % 16 == 0 && (a.lda % 8 == 0 || a.M == 1);
    p.ldc = a.ldc;
    return launch_kernel(k_gemm4<F, NT, Tout>, dim3((a.N + kTileRows - 1) / kTileRows * ranks, (a.M + L::cols - 1) / L::cols), kThreads, ranks,
                         L::bytes, false, s, p, static_cast<Tout*>(a.C));
}

template <int F, int NT> cudaError_t launch_out(const kda_gemm4_args& a, int ranks, cudaStream_t s) {
    return a.c_dtype == KDA_BF16 ? launch<F, NT, bf16>(a, ranks, s) : launch<F, NT, float>(a, ranks, s);
}

template <int F> cudaError_t launch_cols(const kda_gemm4_args& a, int ranks, cudaStream_t s) {
    if (a.M <= 8) return launch_out<F, 1>(a, ranks, s);
    if (a.M <= 16) return launch_out<F, 2>(a, ranks, s);
    if (a.M <= 32) return launch_out<F, 4>(a, ranks, s);
    return launch_out<F, 8>(a, ranks, s);
}

// ------------------------------------------------------------------ block-scaled tensor cores
struct Gemm4Tc {
    int M, N, K, epi, ranks;
    const uint8_t *codes, *w_scales, *b_scales;
    const bf16* a;
    int64_t lda, ldc;
    int* d_status;
};

template <int N, typename Tout>
__global__ void __launch_bounds__(fewtc::kThreads, fewtc::Shape<N>::per_sm) k_gemm4_tc(const __grid_constant__ fewtc::Maps maps, const Gemm4Tc p,
                                                                                      Tout* __restrict__ out) {
    extern __shared__ uint8_t smem_raw[];
    __shared__ fewtc::Barriers bar;
    const uint32_t raw = smem_addr(smem_raw);
    uint8_t* smem = smem_raw + (((raw + 1023u) & ~1023u) - raw);
    const int rank = blockIdx.x % p.ranks, row0 = blockIdx.x / p.ranks * kTileRows;
    constexpr int kTokens = fewtc::Shape<N>::tokens;
    const int c0 = blockIdx.y * kTokens, n = min(kTokens, p.M - c0);
    fewtc::start<N>(bar);
    fewtc::Tile t;
    t.w = &maps.w, t.b = &maps.b;
    t.row0 = row0, t.row64 = row0 + 64, t.token0 = c0;
    t.w_scales = p.w_scales, t.b_scales = p.b_scales, t.last_row = p.N - 1, t.last_token = p.M - 1, t.K = p.K;
    slice_of(p.K, rank, p.ranks, t.k0, t.k1);
    fewtc::Counters count;
    float* red = reinterpret_cast<float*>(smem);
    fewtc::product<N>(smem, bar, t, count, red);
    if (p.ranks > 1) cooperative_groups::this_cluster().sync();
    int r0, r1;
    fewtc::rows_of(rank, p.ranks, r0, r1);
    const int share = (r1 - r0) / 4;
    for (int i = threadIdx.x; i < n * share; i += fewtc::kThreads) {
        const int c = i / share, r = r0 + i % share * 4, left = p.N - row0 - r;
        if (left <= 0) continue;
        const float4 q = fewtc::joined4(red, p.ranks, c, r);
        float v[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int64_t row = row0 + r + j;
            if (isnan(v[j]) && j < left)
                v[j] = fewtc::direct(p.codes + row * (p.K / 2), p.w_scales + row * (p.K / 32), p.a + (int64_t)(c0 + c) * p.lda, p.K);
            if (p.epi != KDA_EPI_NONE) v[j] = (p.epi == KDA_EPI_DECAY ? -5.0f : 1.0f) / (1.0f + expf(-v[j]));
        }
        Tout* o = out + (int64_t)(c0 + c) * p.ldc + row0 + r;
        if (left >= 4 && reinterpret_cast<uintptr_t>(o) % (4 * sizeof(Tout)) == 0) {
            if constexpr (sizeof(Tout) == 4) {
                *reinterpret_cast<float4*>(o) = make_float4(v[0], v[1], v[2], v[3]);
            } else {
                const __nv_bfloat162 lo = __floats2bfloat162_rn(v[0], v[1]), hi = __floats2bfloat162_rn(v[2], v[3]);
                *reinterpret_cast<uint2*>(o) = make_uint2(*reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi));
            }
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (j < left) o[j] = from_f<Tout>(v[j]);
        }
    }
    release(p.ranks);
    fewtc::finish<N>(bar, p.d_status);
}

template <int N, typename Tout> cudaError_t launch_tc(const kda_gemm4_args& a, cudaStream_t s) {
    using S = fewtc::Shape<N>;
    uint8_t* digits = static_cast<uint8_t*>(a.workspace);
    uint8_t* scales = digits + fewtc::digits_bytes(a.M, a.K);
    const bool wide = reinterpret_cast<uintptr_t>(a.A) % 16 == 0 && (a.lda % 8 == 0 || a.M == 1);
    fewtc::Maps maps;
    if (!fewtc::encode_maps(&maps, a.codes, a.N, digits, a.M, a.K, N)) return cudaErrorInvalidValue;
    if (const cudaError_t e = fewtc::launch_digits(static_cast<const bf16*>(a.A), a.lda, wide, nullptr, 1, a.M, a.K, digits, scales, s)) return e;
    const int64_t tiles = (a.N + kTileRows - 1) / kTileRows, blocks = (a.M + S::tokens - 1) / S::tokens;
    Gemm4Tc p;
    p.M = a.M, p.N = a.N, p.K = a.K, p.epi = a.epilogue;
    p.ranks = fewtc::cluster_ranks(tiles * blocks, a.K, S::per_sm, 8);
    p.w_scales = static_cast<const uint8_t*>(a.scales), p.b_scales = scales, p.codes = a.codes;
    p.a = static_cast<const bf16*>(a.A), p.lda = a.lda, p.ldc = a.ldc, p.d_status = a.d_status;
    return launch_kernel(k_gemm4_tc<N, Tout>, dim3(tiles * p.ranks, blocks), fewtc::kThreads, p.ranks, S::smem, true, s, maps, p,
                         static_cast<Tout*>(a.C));
}

template <int N> cudaError_t launch_tc_out(const kda_gemm4_args& a, cudaStream_t s) {
    return a.c_dtype == KDA_BF16 ? launch_tc<N, bf16>(a, s) : launch_tc<N, float>(a, s);
}

}  // namespace

size_t gemm4_workspace(const kda_gemm4_args& a) {
    return a.format == KDA_WEIGHT_E2M1 ? fewtc::digits_bytes(a.M, a.K) + fewtc::digit_scales_bytes(a.M, a.K) : 0;
}

cudaError_t launch_gemm4(const kda_gemm4_args& a, cudaStream_t s) {
    if (a.format == KDA_WEIGHT_E2M1) {
        if (a.M <= 2) return launch_tc_out<16>(a, s);
        if (a.M <= 4) return launch_tc_out<32>(a, s);
        if (a.M <= 8) return launch_tc_out<64>(a, s);
        if (a.M <= 16) return launch_tc_out<128>(a, s);
        return launch_tc_out<256>(a, s);
    }
    const int64_t tiles = (int64_t)((a.N + kTileRows - 1) / kTileRows) * ((a.M + 63) / 64);
    const int ranks = cluster_ranks(tiles, a.K);
    return launch_cols<KDA_WEIGHT_INT4>(a, ranks, s);
}

}  // namespace kda
