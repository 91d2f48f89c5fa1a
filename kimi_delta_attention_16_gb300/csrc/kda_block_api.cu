// kda_block_api.cu -- the C entry points of the operators around the layer (declared in
// include/kda.h): argument checks, workspace sizing and launch sequencing on the caller's stream.
// Nothing here allocates device memory or synchronises, and nothing throws.
#include "kda_api_util.cuh"
#include "kda_block.cuh"

namespace {

using namespace kda;

constexpr int kMaxWidth = 32768;  // channels of a layer norm row (they live in one block's registers)

cudaStream_t cu_stream(kda_stream_t s) { return reinterpret_cast<cudaStream_t>(s); }

// Bytes from the first to past the last element of [M] rows of C elements.
size_t rows_bytes(int64_t M, int64_t stride, int64_t C, size_t esize) {
    return M > 0 ? ((size_t)(M - 1) * (size_t)stride + (size_t)C) * esize : 0;
}

// A row tensor: non-NULL, aligned to its element, rows at least C apart.  (size_t)M * stride must
// stay far inside 63 bits.
kda_status check_plain_rows(const void* p, int64_t M, int64_t stride, int64_t C, size_t esize, const char* name) {
    if (!p) return fail(KDA_ERR_INVALID_ARG, "%s is NULL", name);
    if (!aligned(p, esize)) return fail(KDA_ERR_INVALID_ARG, "%s is not aligned to its element", name);
    if (stride < C)
        return fail(KDA_ERR_INVALID_ARG, "%s row stride %lld < %lld", name, (long long)stride, (long long)C);
    if (M > 1 && stride > ((int64_t)1 << 59) / M)
        return fail(KDA_ERR_UNSUPPORTED, "%s is too large (%lld rows %lld apart)", name, (long long)M, (long long)stride);
    return KDA_OK;
}

kda_status check_f32(const float* p, const char* name) {
    if (p && !aligned(p, 4)) return fail(KDA_ERR_INVALID_ARG, "%s is not aligned to its element", name);
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

kda_status check_workspace(const void* ws, size_t have, size_t need) {
    if (need == 0) return KDA_OK;
    if (!ws) return fail(KDA_ERR_WORKSPACE, "workspace is NULL (%zu bytes needed)", need);
    if (have < need) return fail(KDA_ERR_WORKSPACE, "workspace has %zu bytes, %zu needed", have, need);
    if (!aligned(ws, 256)) return fail(KDA_ERR_WORKSPACE, "workspace is not 256-byte aligned");
    return KDA_OK;
}

kda_status check_norm_sizes(int64_t M, int C, int io) {
    if (M < 0 || C < 1) return fail(KDA_ERR_INVALID_ARG, "bad sizes M=%lld C=%d", (long long)M, C);
    if (C > kMaxWidth) return fail(KDA_ERR_UNSUPPORTED, "C=%d above %d", C, kMaxWidth);
    if (!valid_dtype(io)) return fail(KDA_ERR_INVALID_ARG, "unknown dtype %d", io);
    return KDA_OK;
}

int64_t blocks32(int C) { return (C + KDA_PACK8_BLOCK - 1) / KDA_PACK8_BLOCK; }

}  // namespace

extern "C" {

kda_status kda_layer_norm(const kda_norm_args* a, kda_stream_t stream) {
    if (!a) return fail(KDA_ERR_INVALID_ARG, "args is NULL");
    kda_status st;
    if ((st = check_norm_sizes(a->M, a->C, a->io))) return st;
    if (a->M == 0) return ok();
    const size_t es = dsize(a->io);
    const int64_t xs = a->x_stride ? a->x_stride : a->C, ys = a->y_stride ? a->y_stride : a->C;
    if ((st = check_plain_rows(a->x, a->M, xs, a->C, es, "x")) || (st = check_plain_rows(a->y, a->M, ys, a->C, es, "y")) ||
        (st = check_f32(a->weight, "weight")) || (st = check_f32(a->bias, "bias")) || (st = check_f32(a->stats, "stats")))
        return st;
    const size_t cb = (size_t)a->C * 4;
    const Span outs[] = {{a->y, rows_bytes(a->M, ys, a->C, es), "y"}, {a->stats, (size_t)a->M * 8, "stats"}};
    const Span ins[] = {{a->x, rows_bytes(a->M, xs, a->C, es), "x"}, {a->weight, cb, "weight"}, {a->bias, cb, "bias"}};
    if ((st = check_overlaps(outs, ins))) return st;
    if (const cudaError_t e = launch_layer_norm(*a, cu_stream(stream))) return cuda_fail(e, "layer norm");
    return ok();
}

kda_status kda_layer_norm_backward_workspace_size(const kda_norm_backward_args* a, size_t* bytes) {
    if (!bytes) return fail(KDA_ERR_INVALID_ARG, "bytes is NULL");
    *bytes = 0;
    if (!a) return fail(KDA_ERR_INVALID_ARG, "args is NULL");
    if (kda_status st = check_norm_sizes(a->M, a->C, a->io)) return st;
    *bytes = norm_backward_plan(*a).workspace;
    return ok();
}

kda_status kda_layer_norm_backward(const kda_norm_backward_args* a, kda_stream_t stream) {
    if (!a) return fail(KDA_ERR_INVALID_ARG, "args is NULL");
    kda_status st;
    if ((st = check_norm_sizes(a->M, a->C, a->io))) return st;
    if ((st = check_f32(a->weight, "weight")) || (st = check_f32(a->dweight, "dweight")) ||
        (st = check_f32(a->dbias, "dbias")))
        return st;
    const size_t es = dsize(a->io), cb = (size_t)a->C * 4;
    if (a->M == 0) {  // no rows: the parameters' gradients are zero
        cudaError_t e = cudaSuccess;
        if (a->dweight) e = cudaMemsetAsync(a->dweight, 0, cb, cu_stream(stream));
        if (!e && a->dbias) e = cudaMemsetAsync(a->dbias, 0, cb, cu_stream(stream));
        return e ? cuda_fail(e, "layer norm backward") : ok();
    }
    const bool x8 = a->x_scales != nullptr;
    const int64_t dys = a->dy_stride ? a->dy_stride : a->C, dxs = a->dx_stride ? a->dx_stride : a->C;
    const int64_t xs = x8 ? a->C : (a->x_stride ? a->x_stride : a->C);
    if ((st = check_plain_rows(a->dy, a->M, dys, a->C, es, "dy")) ||
        (st = check_plain_rows(a->x, a->M, xs, a->C, x8 ? 1 : es, "x")) ||
        (st = check_plain_rows(a->dx, a->M, dxs, a->C, es, "dx")))
        return st;
    if (!a->stats) return fail(KDA_ERR_INVALID_ARG, "stats is NULL");
    if ((st = check_f32(a->stats, "stats"))) return st;
    const NormBackwardPlan p = norm_backward_plan(*a);
    if ((st = check_workspace(a->workspace, a->workspace_bytes, p.workspace))) return st;
    const Span outs[] = {{a->dx, rows_bytes(a->M, dxs, a->C, es), "dx"}, {a->dweight, cb, "dweight"},
                         {a->dbias, cb, "dbias"}, {a->workspace, p.workspace, "workspace"}};
    const Span ins[] = {{a->dy, rows_bytes(a->M, dys, a->C, es), "dy"}, {a->x, rows_bytes(a->M, xs, a->C, x8 ? 1 : es), "x"},
                        {a->x_scales, (size_t)(a->M * blocks32(a->C)), "x_scales"}, {a->stats, (size_t)a->M * 8, "stats"},
                        {a->weight, cb, "weight"}};
    if ((st = check_overlaps(outs, ins))) return st;
    if (const cudaError_t e = launch_layer_norm_backward(*a, p, cu_stream(stream)))
        return cuda_fail(e, "layer norm backward");
    return ok();
}

static kda_status check_pack8(const void* x, int64_t xs, int dtype, int64_t M, int C, const uint8_t* codes,
                              const uint8_t* scales) {
    if (M < 0 || C < 1) return fail(KDA_ERR_INVALID_ARG, "bad sizes M=%lld C=%d", (long long)M, C);
    if (!valid_dtype(dtype)) return fail(KDA_ERR_INVALID_ARG, "unknown dtype %d", dtype);
    if (M == 0) return KDA_OK;
    const size_t es = dsize((kda_dtype)dtype);
    if (kda_status st = check_plain_rows(x, M, xs, C, es, "x")) return st;
    if (!codes || !scales) return fail(KDA_ERR_INVALID_ARG, "codes and scales must be non-NULL");
    const Span all[] = {{x, rows_bytes(M, xs, C, es), "x"}, {codes, (size_t)M * C, "codes"},
                        {scales, (size_t)(M * blocks32(C)), "scales"}};
    const Span none[] = {{nullptr, 0, ""}};
    return check_overlaps(all, none);
}

kda_status kda_pack8(const void* x, int64_t x_stride, kda_dtype dtype, int64_t M, int C, uint8_t* codes,
                     uint8_t* scales, kda_stream_t stream) {
    const int64_t xs = x_stride ? x_stride : C;
    if (kda_status st = check_pack8(x, xs, dtype, M, C, codes, scales)) return st;
    if (M == 0) return ok();
    if (const cudaError_t e = launch_pack8(x, xs, dtype, M, C, codes, scales, cu_stream(stream)))
        return cuda_fail(e, "pack8");
    return ok();
}

kda_status kda_unpack8(const uint8_t* codes, const uint8_t* scales, int64_t M, int C, void* x, int64_t x_stride,
                       kda_dtype dtype, kda_stream_t stream) {
    const int64_t xs = x_stride ? x_stride : C;
    if (kda_status st = check_pack8(x, xs, dtype, M, C, codes, scales)) return st;
    if (M == 0) return ok();
    if (const cudaError_t e = launch_unpack8(codes, scales, M, C, x, xs, dtype, cu_stream(stream)))
        return cuda_fail(e, "unpack8");
    return ok();
}

}  // extern "C"
