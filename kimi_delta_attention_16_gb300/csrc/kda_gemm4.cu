// kda_gemm4.cu -- C[M][N] = epilogue(A[M][K] . W[N][K]^T) for few rows of A and weights in 4 bits
// (e2m1 or offset integers under one scale per group): the projections of a decode step.
//
// What a call has to read is N K / 2 bytes of codes and their scales.  e2m1 weights go through the block-scaled tensor
// cores (kda_few_tc.cuh): a CTA takes 128 of the N outputs for some tokens, a cluster splits K.  Integer codes go
// through registers (kda_few.cuh).
//
// Figures here are per call in a captured graph of calls in a row, weights from HBM, columns included.  e2m1, 12,288 x 7,168: 1 row 13 us
// (3.7 TB/s), 32 rows 19 us; 256 rows (kda_widen_tc.cuh) 47 us.  One row is bound by the chain of two launches, first bytes and
// join; 32 rows have 96 CTAs for 152 SMs.  Integer codes, 160,000 x 7,168, 16 rows 185 us (3.2 TB/s): latency of three warps per
// scheduler (issue 45 %, tensor pipe 32 %, HBM 37 %); every 32 rows more read and take apart the codes again (256 x 12,288 x 7,168: 185 us).
#include "kda_few.cuh"
#include "kda_few_tc.cuh"
#include "kda_serve.cuh"
#include "kda_widen_tc.cuh"

namespace kda {

namespace {

using namespace few;

// ------------------------------------------------------------------ integer codes
struct Gemm4 {
    Weights w;
    Columns x;
    int M, N, K, epi, ks, group;
    int64_t ldc;
    const bf16* a;
    int64_t lda;
};

__device__ __forceinline__ float apply(int epi, float v) {
    return epi == KDA_EPI_NONE ? v : (epi == KDA_EPI_DECAY ? -5.0f : 1.0f) / (1.0f + expf(-v));
}

// A CTA takes an equal share of the tiles of 32 rows, 12 / ks at a time (8 / ks where more scales leave room for 8 warps'
// rings only; 160,000 x 7,168, 16 rows: 185 us, 209 with 8).
constexpr int warps_for(int scale_row) { return scale_row <= 8 ? 12 : 8; }

template <int NT, int GS, int SB> __global__ void __launch_bounds__(32 * warps_for(GS * SB), 1) k_gemm4(const Gemm4 p, void* __restrict__ out, bool out32) {
    using L = Layout<warps_for(GS * SB), NT, GS, SB>;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ int of[L::cols];
    const int c0 = blockIdx.y * L::cols, n = min(L::cols, p.M - c0), per = L::W / p.ks;
    const int tiles = (p.N + kRows - 1) / kRows;
    const int first = (int)((int64_t)tiles * blockIdx.x / gridDim.x), last = (int)((int64_t)tiles * (blockIdx.x + 1) / gridDim.x);
    if (threadIdx.x < L::cols) of[threadIdx.x] = c0 + threadIdx.x;
    __syncthreads();
    wait_for_kernel_before();  // the columns
    const auto row_of = [&](int pass, int tile, int r) -> int64_t {
        const int at = first + pass * per + tile;
        return at < last ? min(at * kRows + r, p.N - 1) : -1;
    };
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    products<L>(smem, p.w, p.x, p.K, of, n, p.ks, (last - first + per - 1) / per, row_of, [&](int pass, const float (&acc)[2][NT][4]) {
        const int at = first + pass * per + warp / p.ks;
        if (warp % p.ks || at >= last) return;
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
            for (int c = 0; c < NT; ++c)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int col = 8 * c + 2 * t + (j & 1), row = at * kRows + 16 * u + g + 8 * (j >> 1);
                    if (col >= n || row >= p.N) continue;
                    float v = acc[u][c][j];
                    if (!isfinite(v))
                        v = direct(p.w.codes + (int64_t)row * (p.K / 2), p.w.scales + (int64_t)row * (p.K / p.group) * SB, SB, p.group,
                                   p.a + (int64_t)(c0 + col) * p.lda, p.K);
                    v = apply(p.epi, v);
                    const int64_t o = (int64_t)(c0 + col) * p.ldc + row;
                    if (out32) static_cast<float*>(out)[o] = v; else static_cast<bf16*>(out)[o] = from_f<bf16>(v);
                }
    });
}

template <int NT, int GS, int SB> cudaError_t launch(const kda_gemm4_args& a, cudaStream_t s) {
    using L = Layout<warps_for(GS * SB), NT, GS, SB>;
    const Columns columns = columns_at(a.workspace, a.M, a.K);
    const bool wide = reinterpret_cast<uintptr_t>(a.A) % 16 == 0 && (a.lda % 8 == 0 || a.M == 1);
    if (const cudaError_t e = launch_halves(static_cast<const bf16*>(a.A), a.lda, wide, a.M, a.K, a.group, columns, s)) return e;
    Gemm4 p;
    p.w = Weights{a.codes, static_cast<const uint8_t*>(a.scales)};
    p.x = columns;
    p.M = a.M, p.N = a.N, p.K = a.K, p.epi = a.epilogue, p.ldc = a.ldc, p.group = a.group;
    p.a = static_cast<const bf16*>(a.A), p.lda = a.lda;
    const int tiles = (a.N + kRows - 1) / kRows, blocks = (a.M + L::cols - 1) / L::cols;
    const Split split = split_rows<L>(tiles, blocks, a.K);
    p.ks = split.ks;
    return launch_kernel(k_gemm4<NT, GS, SB>, dim3(split.ctas, blocks), L::threads, 1, L::bytes, true, s, p, a.C, a.c_dtype == KDA_FP32);
}

template <int NT, int SB> cudaError_t launch_group(const kda_gemm4_args& a, cudaStream_t s) {
    return a.group == 32 ? launch<NT, 8, SB>(a, s) : a.group == 64 ? launch<NT, 4, SB>(a, s) : launch<NT, 2, SB>(a, s);
}
template <int NT> cudaError_t launch_scales(const kda_gemm4_args& a, cudaStream_t s) {
    return a.scale_dtype == KDA_BF16 ? launch_group<NT, 2>(a, s) : launch_group<NT, 4>(a, s);
}

// ------------------------------------------------------------------ block-scaled tensor cores
struct Gemm4Tc {
    int M, N, K, epi, ranks;
    const uint8_t *codes, *w_scales, *b_scales;
    const bf16* a;
    int64_t lda, ldc;
    int* d_status;
};

// The part of a tile's joined sums that this rank writes: tokens [c0, c0 + n).  What came out as NaN or infinite is
// computed again from the operands as they were given.
template <int Threads, typename Tout>
__device__ __forceinline__ void put_tile(const Gemm4Tc& p, const float* red, int rank, int row0, int c0, int n, Tout* __restrict__ out) {
    int r0, r1;
    fewtc::rows_of(rank, p.ranks, r0, r1);
    const int share = (r1 - r0) / 4;
    for (int i = threadIdx.x; i < n * share; i += Threads) {
        const int c = i / share, r = r0 + i % share * 4, left = p.N - row0 - r;
        if (left <= 0) continue;
        const float4 q = fewtc::joined4(red, p.ranks, c, r);
        float v[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int64_t row = row0 + r + j;
            if (!isfinite(v[j]) && j < left)
                v[j] = fewtc::direct(p.codes + row * (p.K / 2), p.w_scales + row * (p.K / 32), p.a + (int64_t)(c0 + c) * p.lda, p.K);
            v[j] = apply(p.epi, v[j]);
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
}

template <int N, typename Tout>
__global__ void __launch_bounds__(fewtc::kThreads, fewtc::Shape<N>::per_sm) k_gemm4_tc(const __grid_constant__ fewtc::Maps maps, const Gemm4Tc p,
                                                                                      Tout* __restrict__ out) {
    extern __shared__ uint8_t smem_raw[];
    __shared__ fewtc::Barriers bar;
    const uint32_t raw = tc::smem_u32(smem_raw);
    uint8_t* smem = smem_raw + (((raw + 1023u) & ~1023u) - raw);
    const int rank = blockIdx.x % p.ranks, row0 = blockIdx.x / p.ranks * kTileRows;
    constexpr int kTokens = fewtc::Shape<N>::tokens;
    const int c0 = blockIdx.y * kTokens, n = min(kTokens, p.M - c0);
    fewtc::start<N>(bar);
    fewtc::Tile t;
    t.w = &maps.w, t.b = &maps.b;
    t.row0 = row0, t.row64 = row0 + 64, t.token0 = c0;
    t.w_scales = p.w_scales, t.b_scales = p.b_scales, t.last_row = p.N - 1, t.last_token = p.M - 1, t.K = p.K;
    fewtc::slice_of(p.K, rank, p.ranks, t.k0, t.k1);
    fewtc::Counters count;
    float* red = reinterpret_cast<float*>(smem);
    fewtc::product<N>(smem, bar, t, count, red);
    if (p.ranks > 1) cooperative_groups::this_cluster().sync();
    put_tile<fewtc::kThreads>(p, red, rank, row0, c0, n, out);
    if (p.ranks > 1) cooperative_groups::this_cluster().sync(); else __syncthreads();
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

// ------------------------------------------------------------------ many rows
// 12,288 x 7,168: 256 rows 47 us (0.96 PFLOP/s), of which 7 the start and the end of a CTA; 7,168 x 12,288 45.  Two causes of about
// the same weight: 96 and 112 CTAs leave a third and a quarter of the SMs without work (an SM is active for 66 % of the
// kernel's time), and 128 elements take some 1,270 cycles with 128 columns and 1,430 with 256, whose products alone take 1,024:
// the warp that issues them, by clock stamps where the time went, shares its scheduler with four that widen.  (Barriers and
// commits every 64 elements: 53 us, 46 with 128 rows.)
template <int N>
__global__ void __launch_bounds__(widetc::kThreads, 1) k_gemm4_widen(const __grid_constant__ fewtc::Maps maps, const Gemm4Tc p, bf16* __restrict__ out) {
    extern __shared__ uint8_t smem_raw[];
    __shared__ widetc::Barriers bar;
    const uint32_t raw = tc::smem_u32(smem_raw);
    uint8_t* smem = smem_raw + (((raw + 1023u) & ~1023u) - raw);
    const int rank = blockIdx.x % p.ranks, row0 = blockIdx.x / p.ranks * kTileRows, c0 = blockIdx.y * N;
    widetc::start<N>(bar);
    widetc::Tile t;
    t.w = &maps.w, t.x = &maps.b;
    t.row0 = row0, t.c0 = c0, t.scales = p.w_scales, t.last_row = p.N - 1, t.K = p.K;
    fewtc::slice_of(p.K, rank, p.ranks, t.k0, t.k1);
    float* red = reinterpret_cast<float*>(smem);
    widetc::product<N>(smem, bar, t, red);
    if (p.ranks > 1) cooperative_groups::this_cluster().sync();
    put_tile<widetc::kThreads>(p, red, rank, row0, c0, min(N, p.M - c0), out);
    if (p.ranks > 1) cooperative_groups::this_cluster().sync(); else __syncthreads();
    widetc::finish<N>(bar, p.d_status);
}

// The rows of A packed, eight elements in the order in which codes come out of a word.
__global__ void __launch_bounds__(256) k_widen_rows(const bf16* __restrict__ x, int64_t xs, bool wide, int K, uint4* __restrict__ rows) {
    let_next_kernel_begin();
    const int k = (blockIdx.x * 256 + threadIdx.x) * 8;  // K is a multiple of 32
    if (k >= K) return;
    const bf16* row = x + (int64_t)blockIdx.y * xs + k;
    uint32_t v[4];
    if (wide) {
        const uint4 q = *reinterpret_cast<const uint4*>(row);
        v[0] = q.x, v[1] = q.y, v[2] = q.z, v[3] = q.w;
    } else {
        const unsigned short* h = reinterpret_cast<const unsigned short*>(row);
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = h[2 * i] | (uint32_t)h[2 * i + 1] << 16;
    }
    rows[((int64_t)blockIdx.y * K + k) / 8] = make_uint4(__byte_perm(v[0], v[2], 0x5410), __byte_perm(v[0], v[2], 0x7632),
                                                         __byte_perm(v[1], v[3], 0x5410), __byte_perm(v[1], v[3], 0x7632));
}

template <int N> cudaError_t launch_widen(const kda_gemm4_args& a, cudaStream_t s) {
    using S = widetc::Shape<N>;
    const bf16* x = static_cast<const bf16*>(a.A);
    const bool wide = reinterpret_cast<uintptr_t>(x) % 16 == 0 && a.lda % 8 == 0;
    if (const cudaError_t e = launch_kernel(k_widen_rows, dim3((a.K + 2047) / 2048, a.M), 256, 1, 0, false, s, x, a.lda, wide, a.K,
                                            static_cast<uint4*>(a.workspace)))
        return e;
    fewtc::Maps maps;
    if (!encode_tensor_map_2d_as(&maps.w, CU_TENSOR_MAP_DATA_TYPE_UINT8, a.codes, a.K / 2, a.N, a.K / 2, widetc::kCodesK / 2, kTileRows, true) ||
        !encode_tensor_map_2d_as(&maps.b, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, a.workspace, a.K, a.M, 2 * (uint64_t)a.K, widetc::kSubK, N, true))
        return cudaErrorInvalidValue;
    Gemm4Tc p;
    const int tiles = (a.N + kTileRows - 1) / kTileRows, blocks = (a.M + N - 1) / N;
    p.M = a.M, p.N = a.N, p.K = a.K, p.epi = a.epilogue;
    p.ranks = fewtc::cluster_ranks((int64_t)tiles * blocks, a.K, 1, 10, widetc::least_ranks(a.K));
    p.w_scales = static_cast<const uint8_t*>(a.scales), p.b_scales = nullptr, p.codes = a.codes;
    p.a = static_cast<const bf16*>(a.A), p.lda = a.lda, p.ldc = a.ldc, p.d_status = a.d_status;
    return launch_kernel(k_gemm4_widen<N>, dim3(tiles * p.ranks, blocks), widetc::kThreads, p.ranks, S::smem, true, s, maps, p, static_cast<bf16*>(a.C));
}

template <int N> cudaError_t launch_tc_out(const kda_gemm4_args& a, cudaStream_t s) {
    return a.c_dtype == KDA_BF16 ? launch_tc<N, bf16>(a, s) : launch_tc<N, float>(a, s);
}

}  // namespace

size_t gemm4_workspace(const kda_gemm4_args& a) {
    return a.format == KDA_WEIGHT_E2M1 ? fewtc::digits_bytes(a.M, a.K) + fewtc::digit_scales_bytes(a.M, a.K) : columns_bytes(a.M, a.K, a.group);
}

cudaError_t launch_gemm4(const kda_gemm4_args& a, cudaStream_t s) {
    if (a.format == KDA_WEIGHT_E2M1) {
        // From 97 rows on widened weights, where C is bf16 and a cluster's accumulators take K.  Digits against widened, us: 12,288 x
        // 7,168 64 rows 36 and 36, 96 rows 34 and 37, 128 rows 48 and 38, 256 rows 91 and 47, 512 rows 166 and 87; 7,168 x 12,288 64 rows 25
        // and 36, 96 46 and 36, 128 49 and 37, 256 71 and 45, 512 141 and 74; 7,168 x 7,168 100 rows 35 and 24, 256 rows 49 and 31; 4,000 x
        // 2,048 100 rows 10 and 12, 256 rows 18 and 16.  Small matrices, whose digits' CTAs run all at once, would keep the digits:
        // 1,000 x 1,024 100 rows 7 and 9, 256 rows 9 and 13; 1,024 x 4,096 256 rows 12 and 18.
        if (a.c_dtype == KDA_BF16 && a.M > 96 && widetc::least_ranks(a.K) <= widetc::kMostRanks) return a.M <= 128 ? launch_widen<128>(a, s) : launch_widen<256>(a, s);
        // as few columns as hold all rows, and at most 32 rows' (256 rows of 7,168 x 12,288: 71 us, 82 with 16 rows per CTA, 129 with 8)
        if (a.M <= 2) return launch_tc_out<16>(a, s);
        if (a.M <= 4) return launch_tc_out<32>(a, s);
        if (a.M <= 8) return launch_tc_out<64>(a, s);
        if (a.M <= 16) return launch_tc_out<128>(a, s);
        return launch_tc_out<256>(a, s);
    }
    // 8 columns an instruction: one, two or four of them (160,000 x 7,168 for 16 rows: 301, 185 and 276 us; 1,001 x 1,056 for
    // 5: 6.5, 9.1 and 15.2)
    if (a.M <= 8) return launch_scales<1>(a, s);
    if (a.M <= 16) return launch_scales<2>(a, s);
    return launch_scales<4>(a, s);
}

}  // namespace kda
