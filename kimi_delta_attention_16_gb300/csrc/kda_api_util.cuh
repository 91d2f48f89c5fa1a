// kda_api_util.cuh -- what the C entry points share: the calling thread's error text, and the
// checks of sizes, alignment, overlap and cu_seqlens.  Nothing here throws or allocates.
#pragma once

#include <cstdarg>
#include <cstdio>

#include "kda_internal.cuh"

namespace kda {

// Text of the last error on this host thread (a fixed buffer: setting it cannot fail).
inline thread_local char g_last_error[512] = "";

inline kda_status fail(kda_status code, const char* fmt, ...) {
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(g_last_error, sizeof(g_last_error), fmt, ap);
    va_end(ap);
    return code;
}

inline kda_status cuda_fail(cudaError_t e, const char* where) {
    return fail(KDA_ERR_CUDA, "%s: %s", where, cudaGetErrorString(e));
}

inline kda_status ok() {
    g_last_error[0] = 0;
    return KDA_OK;
}

inline bool supported_d(int D) { return D == 16 || D == 32 || D == 64 || D == 128; }
inline bool valid_dtype(int dt) { return dt == KDA_BF16 || dt == KDA_FP32; }
inline size_t dsize(kda_dtype dt) { return dt == KDA_BF16 ? 2 : 4; }
inline bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
inline size_t round_up(size_t x, size_t a) { return (x + a - 1) / a * a; }

inline bool overlap(const void* a, size_t na, const void* b, size_t nb) {
    if (!a || !b || na == 0 || nb == 0) return false;
    const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    return x < y + nb && y < x + na;
}

// Validates a host copy of cu_seqlens: cu[0] = 0, non-decreasing, cu[N] = T_total.
inline kda_status check_host_cu(const int32_t* cu, int N, int64_t T_total) {
    if (cu[0] != 0) return fail(KDA_ERR_INVALID_ARG, "cu_seqlens[0] = %d, expected 0", cu[0]);
    for (int n = 0; n < N; ++n)
        if (cu[n + 1] < cu[n])
            return fail(KDA_ERR_INVALID_ARG, "cu_seqlens decreases at %d (%d -> %d)", n, cu[n],
                        cu[n + 1]);
    if ((int64_t)cu[N] != T_total)
        return fail(KDA_ERR_INVALID_ARG, "cu_seqlens[N] = %d but T_total = %lld", cu[N],
                    (long long)T_total);
    return KDA_OK;
}

// Row stride and alignment rules for 16-byte vector access of token rows.
inline kda_status check_rows(const void* p, int64_t stride, int64_t min_stride, kda_dtype dt,
                      const char* name) {
    if (stride < min_stride)
        return fail(KDA_ERR_INVALID_ARG, "%s row stride %lld < %lld", name, (long long)stride,
                    (long long)min_stride);
    const int64_t vec = dt == KDA_BF16 ? 8 : 4;
    if (stride % vec)
        return fail(KDA_ERR_INVALID_ARG, "%s row stride %lld is not a multiple of %lld elements",
                    name, (long long)stride, (long long)vec);
    if (!aligned(p, 16)) return fail(KDA_ERR_INVALID_ARG, "%s is not 16-byte aligned", name);
    return KDA_OK;
}

}  // namespace kda
