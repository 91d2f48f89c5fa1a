// kda_block_api.cu -- the C entry points of the operators around the layer (declared in
// include/kda.h): argument checks, workspace sizing and launch sequencing on the caller's stream.
// Nothing here allocates device memory or synchronises, and nothing throws.
#include "kda_api_util.cuh"
#include "kda_block.cuh"

namespace {

using namespace kda;

constexpr int kMaxWidth = 32768;  // channels of a layer norm row (they live in one block's registers)

constexpr int kMaxChannels = 1 << 20;  // channels of the conv and the scan

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

// What the packed-sequence entry points share: sizes, dtype, cu_seqlens.
kda_status check_packed(int N, int C, int64_t T_total, int io, const int32_t* cu, const int32_t* cu_host) {
    if (N < 0 || C < 1 || T_total < 0)
        return fail(KDA_ERR_INVALID_ARG, "bad sizes N=%d C=%d T_total=%lld", N, C, (long long)T_total);
    if (C > kMaxChannels) return fail(KDA_ERR_UNSUPPORTED, "C=%d above %d", C, kMaxChannels);
    if (T_total > 0x7fffffffLL) return fail(KDA_ERR_UNSUPPORTED, "T_total does not fit cu_seqlens (int32)");
    if (!valid_dtype(io)) return fail(KDA_ERR_INVALID_ARG, "unknown dtype %d", io);
    if (N > 0 && !cu) return fail(KDA_ERR_INVALID_ARG, "cu_seqlens is NULL");
    if (cu_host) return check_host_cu(cu_host, N, T_total);
    if (N == 0 && T_total != 0) return fail(KDA_ERR_INVALID_ARG, "N = 0 but T_total = %lld", (long long)T_total);
    return KDA_OK;
}

// Whether a sequence without tokens may be among them (a device-only cu_seqlens is not known here).
bool may_have_empty(int N, const int32_t* cu_host) {
    if (!cu_host) return true;
    for (int n = 0; n < N; ++n)
        if (cu_host[n + 1] == cu_host[n]) return true;
    return false;
}

int64_t stride_or(int64_t s, int64_t d) { return s ? s : d; }

kda_status check_conv_params(const kda_ssm_conv_args& a) {
    if (!a.w) return fail(KDA_ERR_INVALID_ARG, "w is NULL");
    kda_status st;
    if ((st = check_f32(a.w, "w")) || (st = check_f32(a.bias, "bias"))) return st;
    const size_t es = dsize(a.io);
    if ((a.conv_state_in && !aligned(a.conv_state_in, es)) || (a.conv_state_out && !aligned(a.conv_state_out, es)))
        return fail(KDA_ERR_INVALID_ARG, "a conv state is not aligned to its element");
    return KDA_OK;
}

// Sizes and parameters of the scan and the step; T rows of tokens.
kda_status check_ssm_sizes(const kda_ssm_args& a) {
    if (a.Nst != 8 && a.Nst != 16 && a.Nst != 32 && a.Nst != 64)
        return fail(KDA_ERR_UNSUPPORTED, "states per channel Nst=%d not in {8,16,32,64}", a.Nst);
    if (a.G < 1 || a.C < 1 || a.C % a.G)
        return fail(KDA_ERR_INVALID_ARG, "G=%d does not divide C=%d", a.G, a.C);
    return KDA_OK;
}

// The gradients sum dB and dC with one row of blocks per group.
kda_status check_backward_groups(const kda_ssm_args& a) {
    if (a.G > 65535) return fail(KDA_ERR_UNSUPPORTED, "G=%d above 65535", a.G);
    return KDA_OK;
}

size_t state_bytes(const kda_ssm_args& a) { return (size_t)a.N * a.C * a.Nst * sizeof(float); }

kda_status check_ssm_rows(const kda_ssm_args& a, int64_t rows) {
    const size_t es = dsize(a.io);
    const int64_t gn = (int64_t)a.G * a.Nst;
    kda_status st;
    if (!a.A) return fail(KDA_ERR_INVALID_ARG, "A is NULL");
    if ((st = check_plain_rows(a.u, rows, stride_or(a.u_stride, a.C), a.C, es, "u")) ||
        (st = check_plain_rows(a.dt, rows, stride_or(a.dt_stride, a.C), a.C, es, "dt")) ||
        (st = check_plain_rows(a.B, rows, stride_or(a.B_stride, gn), gn, es, "B")) ||
        (st = check_plain_rows(a.Cm, rows, stride_or(a.C_stride, gn), gn, es, "Cm")) ||
        (a.z && (st = check_plain_rows(a.z, rows, stride_or(a.z_stride, a.C), a.C, es, "z"))) ||
        (st = check_f32(a.D, "D")) || (st = check_f32(a.dt_bias, "dt_bias")))
        return st;
    if (!aligned(a.A, 16) || !aligned(a.initial_state, 16) || !aligned(a.final_state, 16))
        return fail(KDA_ERR_INVALID_ARG, "A and the states must be 16-byte aligned");
    return KDA_OK;
}

// The inputs of the scan, the step and the gradients, for the checks of overlap.
struct SsmSpans {
    Span in[9];
};
SsmSpans ssm_inputs(const kda_ssm_args& a, int64_t rows) {
    const size_t es = dsize(a.io), cb = (size_t)a.C * 4;
    const int64_t gn = (int64_t)a.G * a.Nst;
    return SsmSpans{{{a.u, rows_bytes(rows, stride_or(a.u_stride, a.C), a.C, es), "u"},
                     {a.dt, rows_bytes(rows, stride_or(a.dt_stride, a.C), a.C, es), "dt"},
                     {a.B, rows_bytes(rows, stride_or(a.B_stride, gn), gn, es), "B"},
                     {a.Cm, rows_bytes(rows, stride_or(a.C_stride, gn), gn, es), "Cm"},
                     {a.z, rows_bytes(rows, stride_or(a.z_stride, a.C), a.C, es), "z"},
                     {a.A, cb * a.Nst, "A"}, {a.D, cb, "D"}, {a.dt_bias, cb, "dt_bias"},
                     {a.initial_state, state_bytes(a), "initial_state"}}};
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
        (st = check_f32(a->weight, "weight")) || (st = check_f32(a->bias, "bias")))
        return st;
    if (!aligned(a->stats, 8)) return fail(KDA_ERR_INVALID_ARG, "stats is not 8-byte aligned");
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
    if (!aligned(a->stats, 8)) return fail(KDA_ERR_INVALID_ARG, "stats is not 8-byte aligned");
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
    if (C > 1 << 30) return fail(KDA_ERR_UNSUPPORTED, "C=%d above 2^30", C);
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

kda_status kda_ssm_conv(const kda_ssm_conv_args* a, kda_stream_t stream) {
    if (!a) return fail(KDA_ERR_INVALID_ARG, "args is NULL");
    kda_status st;
    if ((st = check_packed(a->N, a->C, a->T_total, a->io, a->cu_seqlens, a->cu_seqlens_host))) return st;
    if (a->N == 0) return ok();
    if ((st = check_conv_params(*a))) return st;
    const size_t es = dsize(a->io), cs = (size_t)a->N * a->C * 3 * es, cb = (size_t)a->C * 4;
    const int64_t xs = stride_or(a->x_stride, a->C), ys = stride_or(a->y_stride, a->C);
    if (a->T_total > 0 && ((st = check_plain_rows(a->x, a->T_total, xs, a->C, es, "x")) ||
                           (st = check_plain_rows(a->y, a->T_total, ys, a->C, es, "y"))))
        return st;
    const Span outs[] = {{a->y, rows_bytes(a->T_total, ys, a->C, es), "y"}, {a->conv_state_out, cs, "conv_state_out"}};
    const Span ins[] = {{a->x, rows_bytes(a->T_total, xs, a->C, es), "x"}, {a->conv_state_in, cs, "conv_state_in"},
                        {a->w, 4 * cb, "w"}, {a->bias, cb, "bias"}};
    if ((st = check_overlaps(outs, ins))) return st;
    cudaStream_t s = cu_stream(stream);
    cudaError_t e;
    if (!a->cu_seqlens_host && (e = launch_check_cu(a->cu_seqlens, a->N, a->T_total, a->d_status, s)))
        return cuda_fail(e, "check cu_seqlens");
    if (a->conv_state_out && may_have_empty(a->N, a->cu_seqlens_host) &&
        (e = launch_empty_sequences(a->cu_seqlens, a->N, a->conv_state_in, a->conv_state_out, cs / a->N, s)))
        return cuda_fail(e, "ssm conv state");
    if (a->T_total > 0 && (e = launch_ssm_conv(*a, s))) return cuda_fail(e, "ssm conv");
    return ok();
}

kda_status kda_ssm_conv_step(const kda_ssm_conv_args* a, kda_stream_t stream) {
    if (!a) return fail(KDA_ERR_INVALID_ARG, "args is NULL");
    if (a->N < 0 || a->C < 1) return fail(KDA_ERR_INVALID_ARG, "bad sizes N=%d C=%d", a->N, a->C);
    if (a->C > kMaxChannels) return fail(KDA_ERR_UNSUPPORTED, "C=%d above %d", a->C, kMaxChannels);
    if (!valid_dtype(a->io)) return fail(KDA_ERR_INVALID_ARG, "unknown dtype %d", (int)a->io);
    if (a->N == 0) return ok();
    kda_status st;
    if ((st = check_conv_params(*a))) return st;
    if (!a->conv_state_out || a->conv_state_in)
        return fail(KDA_ERR_INVALID_ARG, "the step updates conv_state_out in place (non-NULL) and takes no conv_state_in");
    const size_t es = dsize(a->io), cs = (size_t)a->N * a->C * 3 * es, cb = (size_t)a->C * 4;
    const int64_t xs = stride_or(a->x_stride, a->C), ys = stride_or(a->y_stride, a->C);
    if ((st = check_plain_rows(a->x, a->N, xs, a->C, es, "x")) || (st = check_plain_rows(a->y, a->N, ys, a->C, es, "y")))
        return st;
    const Span outs[] = {{a->y, rows_bytes(a->N, ys, a->C, es), "y"}, {a->conv_state_out, cs, "conv_state_out"}};
    const Span ins[] = {{a->x, rows_bytes(a->N, xs, a->C, es), "x"}, {a->w, 4 * cb, "w"}, {a->bias, cb, "bias"}};
    if ((st = check_overlaps(outs, ins))) return st;
    if (const cudaError_t e = launch_ssm_conv_step(*a, cu_stream(stream))) return cuda_fail(e, "ssm conv step");
    return ok();
}

kda_status kda_ssm_conv_backward_workspace_size(const kda_ssm_conv_backward_args* b, size_t* bytes) {
    if (!bytes) return fail(KDA_ERR_INVALID_ARG, "bytes is NULL");
    *bytes = 0;
    if (!b) return fail(KDA_ERR_INVALID_ARG, "args is NULL");
    const kda_ssm_conv_args& f = b->fwd;
    if (f.N < 0 || f.C < 1 || f.T_total < 0 || !valid_dtype(f.io)) return fail(KDA_ERR_INVALID_ARG, "bad sizes or dtype");
    if (f.C > kMaxChannels) return fail(KDA_ERR_UNSUPPORTED, "C=%d above %d", f.C, kMaxChannels);
    if (f.T_total > 0) *bytes = conv_backward_plan(f).workspace;
    return ok();
}

kda_status kda_ssm_conv_backward(const kda_ssm_conv_backward_args* b, kda_stream_t stream) {
    if (!b) return fail(KDA_ERR_INVALID_ARG, "args is NULL");
    const kda_ssm_conv_args& f = b->fwd;
    kda_status st;
    if ((st = check_packed(f.N, f.C, f.T_total, f.io, f.cu_seqlens, f.cu_seqlens_host))) return st;
    if (!b->dw) return fail(KDA_ERR_INVALID_ARG, "dw is NULL");
    if ((st = check_f32(b->dw, "dw")) || (st = check_f32(b->dbias, "dbias")) ||
        (st = check_f32(b->dconv_state_in, "dconv_state_in")))
        return st;
    const size_t es = dsize(f.io), cs = (size_t)f.N * f.C * 3, cb = (size_t)f.C * 4;
    cudaStream_t s = cu_stream(stream);
    cudaError_t e;
    if (f.T_total == 0) {  // no tokens: every gradient is zero
        if ((e = cudaMemsetAsync(b->dw, 0, 4 * cb, s)) || (b->dbias && (e = cudaMemsetAsync(b->dbias, 0, cb, s))) ||
            (b->dconv_state_in && cs && (e = cudaMemsetAsync(b->dconv_state_in, 0, cs * 4, s))))
            return cuda_fail(e, "ssm conv backward");
        return ok();
    }
    if ((st = check_conv_params(f))) return st;
    const int64_t xs = stride_or(f.x_stride, f.C), dys = stride_or(b->dy_stride, f.C), dxs = stride_or(b->dx_stride, f.C);
    if ((st = check_plain_rows(f.x, f.T_total, xs, f.C, es, "x")) ||
        (st = check_plain_rows(b->dy, f.T_total, dys, f.C, es, "dy")) ||
        (st = check_plain_rows(b->dx, f.T_total, dxs, f.C, es, "dx")))
        return st;
    const ConvBackwardPlan p = conv_backward_plan(f);
    if ((st = check_workspace(b->workspace, b->workspace_bytes, p.workspace))) return st;
    const Span outs[] = {{b->dx, rows_bytes(f.T_total, dxs, f.C, es), "dx"}, {b->dw, 4 * cb, "dw"}, {b->dbias, cb, "dbias"},
                         {b->dconv_state_in, cs * 4, "dconv_state_in"}, {b->workspace, p.workspace, "workspace"}};
    const Span ins[] = {{f.x, rows_bytes(f.T_total, xs, f.C, es), "x"}, {b->dy, rows_bytes(f.T_total, dys, f.C, es), "dy"},
                        {f.conv_state_in, cs * es, "conv_state_in"}, {f.w, 4 * cb, "w"}, {f.bias, cb, "bias"}};
    if ((st = check_overlaps(outs, ins))) return st;
    if (!f.cu_seqlens_host && (e = launch_check_cu(f.cu_seqlens, f.N, f.T_total, f.d_status, s)))
        return cuda_fail(e, "check cu_seqlens");
    if (b->dconv_state_in && may_have_empty(f.N, f.cu_seqlens_host) &&
        (e = launch_empty_sequences(f.cu_seqlens, f.N, nullptr, b->dconv_state_in, cs * 4 / f.N, s)))
        return cuda_fail(e, "ssm conv state gradient");
    if ((e = launch_ssm_conv_backward(*b, p, s))) return cuda_fail(e, "ssm conv backward");
    return ok();
}

kda_status kda_ssm_scan_workspace_size(const kda_ssm_args* a, size_t* bytes) {
    if (!bytes) return fail(KDA_ERR_INVALID_ARG, "bytes is NULL");
    *bytes = 0;
    if (!a) return fail(KDA_ERR_INVALID_ARG, "args is NULL");
    if (kda_status st = check_ssm_sizes(*a)) return st;
    if (a->T_total < 0 || a->T_total > 0x7fffffffLL || a->C > kMaxChannels) return fail(KDA_ERR_INVALID_ARG, "bad sizes");
    if (a->T_total > 0) *bytes = scan_plan(*a).workspace;
    return ok();
}

kda_status kda_ssm_scan(const kda_ssm_args* a, kda_stream_t stream) {
    if (!a) return fail(KDA_ERR_INVALID_ARG, "args is NULL");
    kda_status st;
    if ((st = check_packed(a->N, a->C, a->T_total, a->io, a->cu_seqlens, a->cu_seqlens_host)) ||
        (st = check_ssm_sizes(*a)))
        return st;
    if (a->N == 0) return ok();
    const size_t es = dsize(a->io);
    const int64_t ys = stride_or(a->y_stride, a->C);
    ScanPlan p{};
    if (a->T_total > 0) {
        if ((st = check_ssm_rows(*a, a->T_total)) || (st = check_plain_rows(a->y, a->T_total, ys, a->C, es, "y"))) return st;
        p = scan_plan(*a);
        if ((st = check_workspace(a->workspace, a->workspace_bytes, p.workspace))) return st;
    } else if (!aligned(a->initial_state, 16) || !aligned(a->final_state, 16)) {
        return fail(KDA_ERR_INVALID_ARG, "A and the states must be 16-byte aligned");
    }
    const Span outs[] = {{a->y, rows_bytes(a->T_total, ys, a->C, es), "y"}, {a->final_state, state_bytes(*a), "final_state"},
                         {a->workspace, p.workspace, "workspace"}};
    if ((st = check_overlaps(outs, ssm_inputs(*a, a->T_total).in))) return st;
    cudaStream_t s = cu_stream(stream);
    cudaError_t e;
    if (!a->cu_seqlens_host && (e = launch_check_cu(a->cu_seqlens, a->N, a->T_total, a->d_status, s)))
        return cuda_fail(e, "check cu_seqlens");
    if (a->final_state && may_have_empty(a->N, a->cu_seqlens_host) &&
        (e = launch_empty_sequences(a->cu_seqlens, a->N, a->initial_state, a->final_state, state_bytes(*a) / a->N, s)))
        return cuda_fail(e, "ssm final state");
    if (a->T_total > 0 && (e = launch_ssm_scan(*a, p, s))) return cuda_fail(e, "ssm scan");
    return ok();
}

kda_status kda_ssm_step(const kda_ssm_args* a, kda_stream_t stream) {
    if (!a) return fail(KDA_ERR_INVALID_ARG, "args is NULL");
    if (a->N < 0) return fail(KDA_ERR_INVALID_ARG, "bad sizes N=%d", a->N);
    kda_status st;
    if ((st = check_ssm_sizes(*a))) return st;
    if (a->C > kMaxChannels) return fail(KDA_ERR_UNSUPPORTED, "C=%d above %d", a->C, kMaxChannels);
    if (!valid_dtype(a->io)) return fail(KDA_ERR_INVALID_ARG, "unknown dtype %d", (int)a->io);
    if (a->N == 0) return ok();
    if (!a->final_state || a->initial_state)
        return fail(KDA_ERR_INVALID_ARG, "the step updates final_state in place (non-NULL) and takes no initial_state");
    const size_t es = dsize(a->io);
    const int64_t ys = stride_or(a->y_stride, a->C);
    if ((st = check_ssm_rows(*a, a->N)) || (st = check_plain_rows(a->y, a->N, ys, a->C, es, "y"))) return st;
    const int64_t strides[] = {a->u_stride, a->dt_stride, a->z_stride, a->B_stride, a->C_stride, a->y_stride};
    for (int64_t s : strides)
        if (s * (int64_t)es > 0xffffffffLL) return fail(KDA_ERR_UNSUPPORTED, "kda_ssm_step takes row strides below 4 GB");
    const Span outs[] = {{a->y, rows_bytes(a->N, ys, a->C, es), "y"}, {a->final_state, state_bytes(*a), "final_state"}};
    if ((st = check_overlaps(outs, ssm_inputs(*a, a->N).in))) return st;
    if (const cudaError_t e = launch_ssm_step(*a, cu_stream(stream))) return cuda_fail(e, "ssm step");
    return ok();
}

kda_status kda_ssm_backward_workspace_size(const kda_ssm_backward_args* b, size_t* bytes) {
    if (!bytes) return fail(KDA_ERR_INVALID_ARG, "bytes is NULL");
    *bytes = 0;
    if (!b) return fail(KDA_ERR_INVALID_ARG, "args is NULL");
    const kda_ssm_args& f = b->fwd;
    kda_status st;
    if ((st = check_ssm_sizes(f)) || (st = check_backward_groups(f))) return st;
    if (f.T_total < 0 || f.T_total > 0x7fffffffLL || f.C > kMaxChannels) return fail(KDA_ERR_INVALID_ARG, "bad sizes");
    if (f.T_total > 0) *bytes = ssm_backward_plan(f).workspace;
    return ok();
}

kda_status kda_ssm_backward(const kda_ssm_backward_args* b, kda_stream_t stream) {
    if (!b) return fail(KDA_ERR_INVALID_ARG, "args is NULL");
    const kda_ssm_args& f = b->fwd;
    kda_status st;
    if ((st = check_packed(f.N, f.C, f.T_total, f.io, f.cu_seqlens, f.cu_seqlens_host)) || (st = check_ssm_sizes(f)) ||
        (st = check_backward_groups(f)))
        return st;
    const size_t es = dsize(f.io), cb = (size_t)f.C * 4, an = cb * f.Nst, sb = state_bytes(f);
    if (!b->dA) return fail(KDA_ERR_INVALID_ARG, "dA is NULL");
    if (!aligned(b->dA, 4) || !aligned(b->dD, 4) || !aligned(b->ddt_bias, 4) || !aligned(b->dinitial_state, 16) ||
        !aligned(b->d_final_state, 16))
        return fail(KDA_ERR_INVALID_ARG, "dA, dD and ddt_bias must be 4-byte aligned, the states' gradients 16-byte");
    const size_t rb = (size_t)f.T_total * f.C * es, gb = (size_t)f.T_total * f.G * f.Nst * es;
    const int64_t dys = stride_or(b->dy_stride, f.C);
    SsmBackwardPlan p{};
    if (f.T_total > 0) {
        if ((st = check_ssm_rows(f, f.T_total)) || (st = check_plain_rows(b->dy, f.T_total, dys, f.C, es, "dy"))) return st;
        if (!b->du || !b->ddt || !b->dB || !b->dC)
            return fail(KDA_ERR_INVALID_ARG, "du, ddt, dB and dC must be non-NULL");
        if (!aligned(b->du, es) || !aligned(b->ddt, es) || !aligned(b->dB, es) || !aligned(b->dC, es) || !aligned(b->dz, es))
            return fail(KDA_ERR_INVALID_ARG, "a gradient is not aligned to its element");
        if (b->dz && !f.z) return fail(KDA_ERR_INVALID_ARG, "dz wanted but z is NULL");
        p = ssm_backward_plan(f);
        if ((st = check_workspace(b->workspace, b->workspace_bytes, p.workspace))) return st;
    }
    const Span outs[] = {{b->du, rb, "du"}, {b->ddt, rb, "ddt"}, {b->dA, an, "dA"}, {b->dB, gb, "dB"}, {b->dC, gb, "dC"},
                         {b->dD, cb, "dD"}, {b->dz, rb, "dz"}, {b->ddt_bias, cb, "ddt_bias"},
                         {b->dinitial_state, sb, "dinitial_state"}, {b->workspace, p.workspace, "workspace"}};
    if ((st = check_overlaps(outs, ssm_inputs(f, f.T_total).in))) return st;
    const Span more[] = {{b->dy, rows_bytes(f.T_total, dys, f.C, es), "dy"}, {b->d_final_state, sb, "d_final_state"}};
    if ((st = check_overlaps(outs, more))) return st;
    cudaStream_t s = cu_stream(stream);
    cudaError_t e;
    if (f.T_total == 0) {  // no tokens: the final states are the initial ones, every other gradient is zero
        if ((e = cudaMemsetAsync(b->dA, 0, an, s)) || (b->dD && (e = cudaMemsetAsync(b->dD, 0, cb, s))) ||
            (b->ddt_bias && (e = cudaMemsetAsync(b->ddt_bias, 0, cb, s))))
            return cuda_fail(e, "ssm backward");
    }
    if (f.N == 0) return ok();
    if (!f.cu_seqlens_host && (e = launch_check_cu(f.cu_seqlens, f.N, f.T_total, f.d_status, s)))
        return cuda_fail(e, "check cu_seqlens");
    if (b->dinitial_state && may_have_empty(f.N, f.cu_seqlens_host) &&
        (e = launch_empty_sequences(f.cu_seqlens, f.N, b->d_final_state, b->dinitial_state, sb / f.N, s)))
        return cuda_fail(e, "ssm initial state gradient");
    if (f.T_total > 0 && (e = launch_ssm_backward(*b, p, s))) return cuda_fail(e, "ssm backward");
    return ok();
}

}  // extern "C"
