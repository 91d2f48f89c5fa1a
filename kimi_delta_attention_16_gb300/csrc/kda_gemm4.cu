// kda_gemm4.cu -- C[M][N] = epilogue(A[M][K] . W[N][K]^T) for few rows of A and weights in 4 bits
// (e2m1 or offset integers under one scale per group): the projections of a decode step.
//
// What a call has to read is N K / 2 bytes of codes and their scales; kda_few.cuh has the products.
// A CTA takes 128 of the N outputs for up to 64 tokens, a cluster splits K.
#include "kda_few.cuh"
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
    const auto kernel = k_gemm4<F, NT, Tout>;
    if (const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, L::bytes)) return e;
    Gemm4 p;
    p.w = Matrix{a.codes, a.scales, a.format == KDA_WEIGHT_E2M1 ? 0 : a.scale_dtype == KDA_BF16 ? 1 : 2, group_shift(a.group)};
    p.M = a.M, p.N = a.N, p.K = a.K, p.epi = a.epilogue, p.ranks = ranks;
    p.a = static_cast<const bf16*>(a.A), p.lda = a.lda;
    p.wide = reinterpret_cast<uintptr_t>(a.A) % 16 == 0 && (a.lda % 8 == 0 || a.M == 1);
    p.ldc = a.ldc;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = ranks;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((a.N + kTileRows - 1) / kTileRows * ranks, (a.M + L::cols - 1) / L::cols);
    cfg.blockDim = kThreads;
    cfg.dynamicSmemBytes = L::bytes;
    cfg.stream = s;
    cfg.attrs = at;
    cfg.numAttrs = ranks > 1 ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, kernel, p, static_cast<Tout*>(a.C));
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

}  // namespace

cudaError_t launch_gemm4(const kda_gemm4_args& a, cudaStream_t s) {
    const int64_t tiles = (int64_t)((a.N + kTileRows - 1) / kTileRows) * ((a.M + 63) / 64);
    const int ranks = cluster_ranks(tiles, a.K);
    return a.format == KDA_WEIGHT_E2M1 ? launch_cols<KDA_WEIGHT_E2M1>(a, ranks, s) : launch_cols<KDA_WEIGHT_INT4>(a, ranks, s);
}

}  // namespace kda
