// kda_serve_api.cu -- the C entry points of a decode step over few tokens (declared in include/kda.h): argument
// checks and launches on the caller's stream.  Nothing here allocates device memory or synchronises, and nothing throws.
#include "kda_api_util.cuh"
#include "kda_serve.cuh"

namespace {

using namespace kda;

cudaStream_t cu_stream(kda_stream_t s) { return reinterpret_cast<cudaStream_t>(s); }

size_t rows_bytes(int64_t M, int64_t stride, int64_t C, size_t esize) {
    return M > 0 ? ((size_t)(M - 1) * (size_t)stride + (size_t)C) * esize : 0;
}

kda_status check_rows_of(const void* p, int64_t M, int64_t stride, int64_t C, size_t esize, const char* name) {
    if (!p) return fail(KDA_ERR_INVALID_ARG, "%s is NULL", name);
    if (!aligned(p, esize)) return fail(KDA_ERR_INVALID_ARG, "%s is not aligned to its element", name);
    if (stride < C) return fail(KDA_ERR_INVALID_ARG, "%s row stride %lld < %lld", name, (long long)stride, (long long)C);
    if (M > 1 && stride > ((int64_t)1 << 59) / M)
        return fail(KDA_ERR_UNSUPPORTED, "%s is too large (%lld rows %lld apart)", name, (long long)M, (long long)stride);
    return KDA_OK;
}

struct Span {
    const void* p;
    size_t n;
    const char* name;
};
// No output may overlap another output or an input.
template <int NO, int NI> kda_status check_overlaps(const Span (&outs)[NO], const Span (&ins)[NI]) {
    for (int i = 0; i < NO; ++i) {
        for (int j = i + 1; j < NO; ++j)
            if (overlap(outs[i].p, outs[i].n, outs[j].p, outs[j].n))
                return fail(KDA_ERR_INVALID_ARG, "%s overlaps %s", outs[i].name, outs[j].name);
        for (int j = 0; j < NI; ++j)
            if (overlap(outs[i].p, outs[i].n, ins[j].p, ins[j].n))
                return fail(KDA_ERR_INVALID_ARG, "%s overlaps %s", outs[i].name, ins[j].name);
    }
    return KDA_OK;
}

size_t scale_size(int format, int scale_dtype) { return format == KDA_WEIGHT_E2M1 ? 1 : dsize((kda_dtype)scale_dtype); }

// Format, group and the axis that is cut into groups.
kda_status check_format(int format, int group, int scale_dtype, int K, bool bf16_too, const char* axis) {
    if (format == KDA_WEIGHT_BF16 && bf16_too) {
        if (K % 8) return fail(KDA_ERR_UNSUPPORTED, "%s=%d is not a multiple of 8", axis, K);
        return KDA_OK;
    }
    if (format != KDA_WEIGHT_E2M1 && format != KDA_WEIGHT_INT4) return fail(KDA_ERR_INVALID_ARG, "unknown weight format %d", format);
    if (format == KDA_WEIGHT_E2M1 && group != 32) return fail(KDA_ERR_UNSUPPORTED, "e2m1 weights have groups of 32, not %d", group);
    if (group != 32 && group != 64 && group != 128) return fail(KDA_ERR_UNSUPPORTED, "group=%d not in {32,64,128}", group);
    if (format == KDA_WEIGHT_INT4 && !valid_dtype(scale_dtype)) return fail(KDA_ERR_INVALID_ARG, "unknown scale dtype %d", scale_dtype);
    if (K % group) return fail(KDA_ERR_UNSUPPORTED, "%s=%d is not a multiple of the group of %d", axis, K, group);
    return KDA_OK;
}

// One weight tensor of `rows` rows along K.
kda_status check_weight(const void* w, const void* scales, int format, int scale_dtype, const char* name) {
    if (!w) return fail(KDA_ERR_INVALID_ARG, "%s is NULL", name);
    if (!aligned(w, 16)) return fail(KDA_ERR_INVALID_ARG, "%s is not 16-byte aligned", name);
    if (format == KDA_WEIGHT_BF16) return KDA_OK;
    if (!scales) return fail(KDA_ERR_INVALID_ARG, "the scales of %s are NULL", name);
    if (!aligned(scales, scale_size(format, scale_dtype)))
        return fail(KDA_ERR_INVALID_ARG, "the scales of %s are not aligned to their element", name);
    return KDA_OK;
}

size_t weight_size(int64_t rows, int64_t K, int format) { return (size_t)rows * K * (format == KDA_WEIGHT_BF16 ? 4 : 1) / 2; }
size_t scales_size(int64_t rows, int64_t K, int format, int group, int scale_dtype) {
    return format == KDA_WEIGHT_BF16 ? 0 : (size_t)rows * (K / group) * scale_size(format, scale_dtype);
}

kda_status check_pack4(const kda_pack4_args* a) {
    if (!a) return fail(KDA_ERR_INVALID_ARG, "args is NULL");
    if (a->rows < 0 || a->K < 1) return fail(KDA_ERR_INVALID_ARG, "bad sizes rows=%lld K=%d", (long long)a->rows, a->K);
    if (a->K > 1 << 28) return fail(KDA_ERR_UNSUPPORTED, "K=%d above 2^28", a->K);
    if (!valid_dtype(a->w_dtype)) return fail(KDA_ERR_INVALID_ARG, "unknown dtype %d", (int)a->w_dtype);
    kda_status st;
    if ((st = check_format(a->format, a->group, a->scale_dtype, a->K, false, "K"))) return st;
    if (a->rows == 0) return KDA_OK;
    const int64_t ws = a->w_stride ? a->w_stride : a->K;
    if ((st = check_rows_of(a->w, a->rows, ws, a->K, dsize(a->w_dtype), "w")) ||
        (st = check_weight(a->codes, a->scales, a->format, a->scale_dtype, "codes")))
        return st;
    const Span all[] = {{a->w, rows_bytes(a->rows, ws, a->K, dsize(a->w_dtype)), "w"},
                        {a->codes, weight_size(a->rows, a->K, a->format), "codes"},
                        {a->scales, scales_size(a->rows, a->K, a->format, a->group, a->scale_dtype), "scales"}};
    const Span none[] = {{nullptr, 0, ""}};
    return check_overlaps(all, none);
}

kda_status check_gemm4(const kda_gemm4_args* a) {
    if (!a) return fail(KDA_ERR_INVALID_ARG, "args is NULL");
    if (a->M < 0 || a->N < 0 || a->K < 1) return fail(KDA_ERR_INVALID_ARG, "bad sizes M=%d N=%d K=%d", a->M, a->N, a->K);
    if (a->M > 65535 || a->N > 1 << 24 || a->K > 1 << 24)
        return fail(KDA_ERR_UNSUPPORTED, "M=%d above 65535, or N=%d or K=%d above 2^24", a->M, a->N, a->K);
    kda_status st;
    if ((st = check_format(a->format, a->group, a->scale_dtype, a->K, false, "K"))) return st;
    if (!valid_dtype(a->c_dtype)) return fail(KDA_ERR_INVALID_ARG, "unknown dtype %d", (int)a->c_dtype);
    if (a->epilogue < KDA_EPI_NONE || a->epilogue > KDA_EPI_SIGMOID) return fail(KDA_ERR_INVALID_ARG, "unknown epilogue %d", a->epilogue);
    return KDA_OK;
}

kda_status check_workspace(const void* ws, size_t have, size_t need) {
    if (need == 0) return KDA_OK;
    if (!ws) return fail(KDA_ERR_WORKSPACE, "workspace is NULL (%zu bytes needed)", need);
    if (have < need) return fail(KDA_ERR_WORKSPACE, "workspace has %zu bytes, %zu needed", have, need);
    if (!aligned(ws, 256)) return fail(KDA_ERR_WORKSPACE, "workspace is not 256-byte aligned");
    return KDA_OK;
}

kda_status check_moe(const kda_moe_args* a) {
    if (!a) return fail(KDA_ERR_INVALID_ARG, "args is NULL");
    if (a->M < 0 || a->E < 1 || a->D < 1 || a->F < 1)
        return fail(KDA_ERR_INVALID_ARG, "bad sizes M=%d E=%d D=%d F=%d", a->M, a->E, a->D, a->F);
    if (a->top < 1 || a->top > a->E) return fail(KDA_ERR_INVALID_ARG, "top=%d not in [1, E=%d]", a->top, a->E);
    if (a->E > 1024) return fail(KDA_ERR_UNSUPPORTED, "E=%d above 1024", a->E);
    if (a->top > 32) return fail(KDA_ERR_UNSUPPORTED, "top=%d above 32", a->top);
    if ((int64_t)a->M * a->top > 65535) return fail(KDA_ERR_UNSUPPORTED, "M * top = %lld above 65535", (long long)a->M * a->top);
    if (a->D > 1 << 20 || a->F > 1 << 20) return fail(KDA_ERR_UNSUPPORTED, "D=%d or F=%d above 2^20", a->D, a->F);
    if ((int64_t)a->E * 2 * a->F > 1 << 30 || (int64_t)a->E * a->D > 1 << 30)
        return fail(KDA_ERR_UNSUPPORTED, "the experts have more than 2^30 rows (E=%d D=%d F=%d)", a->E, a->D, a->F);
    if (!valid_dtype(a->router_dtype) || !valid_dtype(a->y_dtype)) return fail(KDA_ERR_INVALID_ARG, "unknown dtype");
    if (a->score != KDA_SCORE_SIGMOID && a->score != KDA_SCORE_SOFTMAX) return fail(KDA_ERR_INVALID_ARG, "unknown score %d", a->score);
    if (a->score == KDA_SCORE_SOFTMAX && a->bias) return fail(KDA_ERR_INVALID_ARG, "softmax scores take no bias");
    kda_status st;
    if ((st = check_format(a->format, a->group, a->scale_dtype, a->D, true, "D"))) return st;
    return check_format(a->format, a->group, a->scale_dtype, a->F, true, "F");
}

}  // namespace

extern "C" {

kda_status kda_pack4(const kda_pack4_args* a, kda_stream_t stream) {
    if (kda_status st = check_pack4(a)) return st;
    if (a->rows == 0) return ok();
    if (const cudaError_t e = launch_pack4(*a, cu_stream(stream))) return cuda_fail(e, "pack4");
    return ok();
}

kda_status kda_unpack4(const kda_pack4_args* a, kda_stream_t stream) {
    if (kda_status st = check_pack4(a)) return st;
    if (a->rows == 0) return ok();
    if (const cudaError_t e = launch_unpack4(*a, cu_stream(stream))) return cuda_fail(e, "unpack4");
    return ok();
}

kda_status kda_gemm4_workspace_size(const kda_gemm4_args* a, size_t* bytes) {
    if (!bytes) return fail(KDA_ERR_INVALID_ARG, "bytes is NULL");
    *bytes = 0;
    if (kda_status st = check_gemm4(a)) return st;
    *bytes = a->N ? gemm4_workspace(*a) : 0;
    return ok();
}

kda_status kda_gemm4(const kda_gemm4_args* a, kda_stream_t stream) {
    kda_status st;
    if ((st = check_gemm4(a))) return st;
    if (a->M == 0 || a->N == 0) return ok();
    if ((st = check_rows_of(a->A, a->M, a->lda, a->K, 2, "A")) ||
        (st = check_rows_of(a->C, a->M, a->ldc, a->N, dsize(a->c_dtype), "C")) ||
        (st = check_weight(a->codes, a->scales, a->format, a->scale_dtype, "codes")))
        return st;
    const size_t ws = gemm4_workspace(*a);
    if ((st = check_workspace(a->workspace, a->workspace_bytes, ws))) return st;
    const Span outs[] = {{a->C, rows_bytes(a->M, a->ldc, a->N, dsize(a->c_dtype)), "C"}, {a->workspace, ws, "workspace"}};
    const Span ins[] = {{a->A, rows_bytes(a->M, a->lda, a->K, 2), "A"}, {a->codes, weight_size(a->N, a->K, a->format), "codes"},
                        {a->scales, scales_size(a->N, a->K, a->format, a->group, a->scale_dtype), "scales"}};
    if ((st = check_overlaps(outs, ins))) return st;
    if (!gemm_supported_device()) return fail(KDA_ERR_UNSUPPORTED, "kda_gemm4 needs an sm_103 device");
    if (const cudaError_t e = launch_gemm4(*a, cu_stream(stream))) return cuda_fail(e, "gemm4");
    return ok();
}

kda_status kda_moe_workspace_size(const kda_moe_args* a, size_t* bytes) {
    if (!bytes) return fail(KDA_ERR_INVALID_ARG, "bytes is NULL");
    *bytes = 0;
    if (kda_status st = check_moe(a)) return st;
    *bytes = a->M ? moe_plan(*a).workspace : 0;
    return ok();
}

kda_status kda_moe(const kda_moe_args* a, kda_stream_t stream) {
    kda_status st;
    if ((st = check_moe(a))) return st;
    if (a->M == 0) return ok();
    const int64_t xs = a->x_stride ? a->x_stride : a->D, ys = a->y_stride ? a->y_stride : a->D;
    const size_t rs = dsize(a->router_dtype);
    if ((st = check_rows_of(a->x, a->M, xs, a->D, 2, "x")) || (st = check_rows_of(a->y, a->M, ys, a->D, dsize(a->y_dtype), "y")) ||
        (st = check_rows_of(a->router, a->E, a->D, a->D, rs, "router")) ||
        (st = check_weight(a->w_in, a->w_in_scales, a->format, a->scale_dtype, "w_in")) ||
        (st = check_weight(a->w_out, a->w_out_scales, a->format, a->scale_dtype, "w_out")))
        return st;
    if (!aligned(a->bias, 4) || !aligned(a->ids, 4) || !aligned(a->weights, 4))
        return fail(KDA_ERR_INVALID_ARG, "bias, ids or weights is not aligned to its element");
    const MoePlan p = moe_plan(*a);
    if ((st = check_workspace(a->workspace, a->workspace_bytes, p.workspace))) return st;
    const size_t slots = (size_t)a->M * a->top * 4;
    const int64_t in = (int64_t)a->E * 2 * a->F, out = (int64_t)a->E * a->D;
    const Span outs[] = {{a->y, rows_bytes(a->M, ys, a->D, dsize(a->y_dtype)), "y"}, {a->ids, slots, "ids"},
                         {a->weights, slots, "weights"}, {a->workspace, p.workspace, "workspace"}};
    const Span ins[] = {{a->x, rows_bytes(a->M, xs, a->D, 2), "x"}, {a->router, (size_t)a->E * a->D * rs, "router"},
                        {a->bias, (size_t)a->E * 4, "bias"}, {a->w_in, weight_size(in, a->D, a->format), "w_in"},
                        {a->w_in_scales, scales_size(in, a->D, a->format, a->group, a->scale_dtype), "w_in_scales"},
                        {a->w_out, weight_size(out, a->F, a->format), "w_out"},
                        {a->w_out_scales, scales_size(out, a->F, a->format, a->group, a->scale_dtype), "w_out_scales"}};
    if ((st = check_overlaps(outs, ins))) return st;
    if (!gemm_supported_device()) return fail(KDA_ERR_UNSUPPORTED, "kda_moe needs an sm_103 device");
    if (const cudaError_t e = launch_moe(*a, p, cu_stream(stream))) return cuda_fail(e, "moe");
    return ok();
}

kda_status kda_verify(const kda_verify_args* a, kda_stream_t stream) {
    if (!a) return fail(KDA_ERR_INVALID_ARG, "args is NULL");
    if (a->N < 0 || a->T_total < 0 || a->V < 1)
        return fail(KDA_ERR_INVALID_ARG, "bad sizes N=%d T_total=%lld V=%d", a->N, (long long)a->T_total, a->V);
    if (a->V > 4000000) return fail(KDA_ERR_UNSUPPORTED, "V=%d above 4,000,000", a->V);
    if (a->N > 1 << 24) return fail(KDA_ERR_UNSUPPORTED, "N=%d above 2^24", a->N);
    if (a->T_total > 0x7fffffffLL) return fail(KDA_ERR_UNSUPPORTED, "T_total does not fit cu_seqlens (int32)");
    if (!valid_dtype(a->dtype)) return fail(KDA_ERR_INVALID_ARG, "unknown dtype %d", (int)a->dtype);
    if (a->token_bytes != 4 && a->token_bytes != 8) return fail(KDA_ERR_INVALID_ARG, "token_bytes=%d not 4 or 8", a->token_bytes);
    if (a->N > 0 && !a->cu_seqlens) return fail(KDA_ERR_INVALID_ARG, "cu_seqlens is NULL");
    kda_status st;
    if (a->cu_seqlens_host && (st = check_host_cu(a->cu_seqlens_host, a->N, a->T_total))) return st;
    if (a->N == 0) return a->T_total ? fail(KDA_ERR_INVALID_ARG, "N = 0 but T_total = %lld", (long long)a->T_total) : ok();
    if (!a->accepted || !aligned(a->accepted, 4)) return fail(KDA_ERR_INVALID_ARG, "accepted is NULL or not aligned to its element");
    const size_t es = dsize(a->dtype), tb = (size_t)a->T_total * a->token_bytes;
    const int64_t ps = a->target_stride ? a->target_stride : a->V, qs = a->draft_stride ? a->draft_stride : a->V;
    if (a->T_total > 0) {
        if ((st = check_rows_of(a->target, a->T_total, ps, a->V, es, "target")) ||
            (a->draft && (st = check_rows_of(a->draft, a->T_total, qs, a->V, es, "draft"))) ||
            (st = check_rows_of(a->tokens, a->T_total, 1, 1, a->token_bytes, "tokens")) ||
            (st = check_rows_of(a->out, a->T_total, 1, 1, a->token_bytes, "out")) ||
            (st = check_rows_of(a->u, a->T_total, 1, 1, 4, "u")))
            return st;
    }
    const Span outs[] = {{a->out, tb, "out"}, {a->accepted, (size_t)a->N * 4, "accepted"}};
    const Span ins[] = {{a->target, rows_bytes(a->T_total, ps, a->V, es), "target"},
                        {a->draft, rows_bytes(a->T_total, qs, a->V, es), "draft"}, {a->tokens, tb, "tokens"},
                        {a->u, (size_t)a->T_total * 4, "u"}, {a->cu_seqlens, (size_t)(a->N + 1) * 4, "cu_seqlens"}};
    if ((st = check_overlaps(outs, ins))) return st;
    cudaError_t e;
    if (!a->cu_seqlens_host && (e = launch_check_cu(a->cu_seqlens, a->N, a->T_total, a->d_status, cu_stream(stream))))
        return cuda_fail(e, "check cu_seqlens");
    if ((e = launch_verify(*a, cu_stream(stream)))) return cuda_fail(e, "verify");
    return ok();
}

}  // extern "C"
