"""PyTorch-facing binding of the operators around the layer in a hybrid block: layer norm, 8-bit
storage of activations, and the selective state space scan with its short causal convolution.

Marshalling only, as in ``api``: the arithmetic runs in libkda.so.  Every tensor lives on the
current CUDA device.  Rows may be strided views (the last axis contiguous); outputs and workspace
are allocated on the stream that the call runs on.
"""
from __future__ import annotations

import contextlib
import ctypes
from typing import Optional

import torch
from torch.autograd.function import once_differentiable

from . import _lib
from .api import _DT, KDAError, _cu_pair, _same_cuda_device

SAVED = ("io", "e4m3")  # how a layer keeps its large inputs for its backward pass


@contextlib.contextmanager
def _on(stream, *inputs):
    """The stream of a call as an integer.  With a stream given that is not the current one, what the
    call allocates belongs to that stream, and the inputs are marked as used on it, so that the
    allocator gives neither away before the kernels are done."""
    if stream is None:
        yield torch.cuda.current_stream().cuda_stream
        return
    s = stream if isinstance(stream, torch.cuda.Stream) else torch.cuda.ExternalStream(int(stream))
    if s == torch.cuda.current_stream():
        yield s.cuda_stream
        return
    for t in inputs:
        if t is not None and t.is_cuda:
            t.record_stream(s)
    with torch.cuda.stream(s):
        yield s.cuda_stream


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else t.data_ptr()


def _io(t: torch.Tensor, name: str) -> int:
    if t.dtype not in _DT:
        raise ValueError(f"{name} is {t.dtype}; expected bfloat16 or float32")
    return _DT[t.dtype]


def _rows(t: torch.Tensor, shape, dtype, name: str) -> int:
    """Row stride (elements) of a [M, C] tensor whose rows are dense."""
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must be {tuple(shape)}, got {tuple(t.shape)}")
    if t.dtype != dtype:
        raise ValueError(f"{name} is {t.dtype}, expected {dtype}")
    if t.shape[1] > 1 and t.stride(1) != 1:
        raise ValueError(f"the rows of {name} must be contiguous")
    return t.stride(0) if t.shape[0] > 1 else t.shape[1]


def _dense(t: Optional[torch.Tensor], shape, dtype, name: str) -> None:
    if t is None:
        return
    if tuple(t.shape) != tuple(shape) or t.dtype != dtype or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} tensor of shape {tuple(shape)}, "
                         f"got {t.dtype} {tuple(t.shape)}")


def _check(st: int, where: str) -> None:
    if st:
        raise KDAError(st, where)


def _workspace(size_fn, args, where: str, workspace, device):
    """Fills args.workspace: the caller's buffer, or a new one of the size the library asks for."""
    if workspace is None:
        n = ctypes.c_size_t(0)
        _check(size_fn(ctypes.byref(args), ctypes.byref(n)), where)
        if n.value == 0:
            return None
        workspace = torch.empty(n.value, dtype=torch.uint8, device=device)
    args.workspace = workspace.data_ptr()
    args.workspace_bytes = workspace.numel() * workspace.element_size()
    return workspace


# ------------------------------------------------------------------ layer norm
def kda_layer_norm(x: torch.Tensor, weight: Optional[torch.Tensor] = None, bias: Optional[torch.Tensor] = None, *,
                   eps: float = 1e-5, y: Optional[torch.Tensor] = None, return_stats: bool = False, stream=None):
    """Layer norm over the last axis of x [M, C] (bf16 or fp32, rows may be strided); weight and bias [C] fp32 or
    None.  Returns y (x's dtype), or (y, stats) with return_stats: stats [M, 2] fp32 holds each row's mean and
    1 / sqrt(var + eps), which kda_layer_norm_backward reads.  C is at most 32768."""
    lib = _lib.load()
    if x.dim() != 2:
        raise ValueError(f"expected x [M, C], got {tuple(x.shape)}")
    a = _lib.NormArgs()
    a.M, a.C, a.io = x.shape[0], x.shape[1], _io(x, "x")
    a.x, a.x_stride = x.data_ptr(), _rows(x, x.shape, x.dtype, "x")
    _dense(weight, (a.C,), torch.float32, "weight")
    _dense(bias, (a.C,), torch.float32, "bias")
    _same_cuda_device(x=x, weight=weight, bias=bias, y=y)
    with _on(stream, x, weight, bias, y) as s:
        if y is None:
            y = torch.empty(x.shape, dtype=x.dtype, device=x.device)
        stats = torch.empty((a.M, 2), dtype=torch.float32, device=x.device) if return_stats else None
        a.weight, a.bias, a.eps = _ptr(weight), _ptr(bias), float(eps)
        a.y, a.y_stride, a.stats = y.data_ptr(), _rows(y, x.shape, x.dtype, "y"), _ptr(stats)
        _check(lib.kda_layer_norm(ctypes.byref(a), s), "kda_layer_norm")
    return (y, stats) if return_stats else y


def kda_layer_norm_backward(dy: torch.Tensor, x: torch.Tensor, stats: torch.Tensor,
                            weight: Optional[torch.Tensor] = None, *, x_scales: Optional[torch.Tensor] = None,
                            param_grads: bool = True, workspace: Optional[torch.Tensor] = None, stream=None) -> dict:
    """Gradients of sum(dy * y) of one kda_layer_norm call: a dict of dx (dy's dtype) and, with param_grads, dweight
    and dbias [C] fp32 (summed in a fixed order).  x is the forward's input, or its 8-bit codes with x_scales given
    (the pair kda_pack8 returns), which the kernel reads directly; stats come from the forward."""
    lib = _lib.load()
    if dy.dim() != 2:
        raise ValueError(f"expected dy [M, C], got {tuple(dy.shape)}")
    a = _lib.NormBackwardArgs()
    a.M, a.C, a.io = dy.shape[0], dy.shape[1], _io(dy, "dy")
    a.dy, a.dy_stride = dy.data_ptr(), _rows(dy, dy.shape, dy.dtype, "dy")
    if x_scales is None:
        a.x_stride = _rows(x, dy.shape, dy.dtype, "x")
    else:
        _dense(x, dy.shape, torch.uint8, "x (8-bit codes)")
        _dense(x_scales, (a.M, -(-a.C // _lib.KDA_PACK8_BLOCK)), torch.uint8, "x_scales")
    a.x, a.x_scales = x.data_ptr(), _ptr(x_scales)
    _dense(stats, (a.M, 2), torch.float32, "stats")
    _dense(weight, (a.C,), torch.float32, "weight")
    _same_cuda_device(dy=dy, x=x, stats=stats, weight=weight, x_scales=x_scales, workspace=workspace)
    dev = dy.device
    with _on(stream, dy, x, stats, weight, x_scales, workspace) as s:
        res = {"dx": torch.empty(dy.shape, dtype=dy.dtype, device=dev)}
        if param_grads:
            res["dweight"] = torch.empty((a.C,), dtype=torch.float32, device=dev)
            res["dbias"] = torch.empty((a.C,), dtype=torch.float32, device=dev)
        a.stats, a.weight, a.dx = stats.data_ptr(), _ptr(weight), res["dx"].data_ptr()
        a.dweight, a.dbias = _ptr(res.get("dweight")), _ptr(res.get("dbias"))
        workspace = _workspace(lib.kda_layer_norm_backward_workspace_size, a, "kda_layer_norm_backward_workspace_size",
                               workspace, dev)
        _check(lib.kda_layer_norm_backward(ctypes.byref(a), s), "kda_layer_norm_backward")
    return res


# ------------------------------------------------------------------ activations in 8 bits
def kda_pack8(x: torch.Tensor, *, stream=None):
    """x [M, C] (bf16 or fp32, rows may be strided) in 8 bits: (codes [M, C] uint8, scales [M, ceil(C / 32)] uint8).
    Each block of 32 channels is stored as e4m3 under the smallest power of two that keeps its largest magnitude
    within 448; scales hold the exponent + 127.  NaN and infinities come back as NaN."""
    lib = _lib.load()
    if x.dim() != 2:
        raise ValueError(f"expected x [M, C], got {tuple(x.shape)}")
    M, C = x.shape
    io, xs = _io(x, "x"), _rows(x, x.shape, x.dtype, "x")
    _same_cuda_device(x=x)
    with _on(stream, x) as s:
        codes = torch.empty((M, C), dtype=torch.uint8, device=x.device)
        scales = torch.empty((M, -(-C // _lib.KDA_PACK8_BLOCK)), dtype=torch.uint8, device=x.device)
        _check(lib.kda_pack8(x.data_ptr(), xs, io, M, C, codes.data_ptr(), scales.data_ptr(), s), "kda_pack8")
    return codes, scales


def kda_unpack8(codes: torch.Tensor, scales: torch.Tensor, *, dtype=torch.bfloat16, out: Optional[torch.Tensor] = None,
                stream=None) -> torch.Tensor:
    """The values that kda_pack8's codes and scales stand for, [M, C] in dtype (exact in bf16 and fp32 wherever the
    value itself is a normal number)."""
    lib = _lib.load()
    if codes.dim() != 2:
        raise ValueError(f"expected codes [M, C], got {tuple(codes.shape)}")
    M, C = codes.shape
    _dense(codes, (M, C), torch.uint8, "codes")
    _dense(scales, (M, -(-C // _lib.KDA_PACK8_BLOCK)), torch.uint8, "scales")
    _same_cuda_device(codes=codes, scales=scales, out=out)
    with _on(stream, codes, scales, out) as s:
        if out is None:
            out = torch.empty((M, C), dtype=dtype, device=codes.device)
        io, xs = _io(out, "out"), _rows(out, (M, C), out.dtype, "out")
        _check(lib.kda_unpack8(codes.data_ptr(), scales.data_ptr(), M, C, out.data_ptr(), xs, io, s), "kda_unpack8")
    return out


def _check_saved(saved: str) -> None:
    if saved not in SAVED:
        raise ValueError(f"saved must be one of {SAVED}, got {saved!r}")


class _NormLayer(torch.autograd.Function):
    """kda_layer_norm forward, kda_layer_norm_backward backward."""

    @staticmethod
    def forward(ctx, x, weight, bias, eps, saved):
        y, stats = kda_layer_norm(x, weight, bias, eps=eps, return_stats=True)
        kept = kda_pack8(x) if saved == "e4m3" else (x, None)
        ctx.save_for_backward(*kept, stats, weight)
        ctx.has_bias = bias is not None
        return y

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        x, scales, stats, weight = ctx.saved_tensors
        want = ctx.needs_input_grad
        g = kda_layer_norm_backward(dy.contiguous(), x, stats, weight, x_scales=scales, param_grads=want[1] or want[2])
        return (g["dx"] if want[0] else None, g["dweight"] if want[1] else None, g["dbias"] if want[2] else None,
                None, None)


def kda_norm_layer(x: torch.Tensor, weight: Optional[torch.Tensor] = None, bias: Optional[torch.Tensor] = None, *,
                   eps: float = 1e-5, saved: str = "io") -> torch.Tensor:
    """Layer norm of x [M, C] as a differentiable PyTorch operation.  saved="e4m3" keeps x in 8 bits for the backward
    pass (a little over half the memory of bf16): the gradients are then those at the rounded x, with the exact
    mean and deviation."""
    _check_saved(saved)
    return _NormLayer.apply(x, weight, bias, float(eps), saved)


# ------------------------------------------------------------------ the selective scan's short convolution
def _param(t: Optional[torch.Tensor], shape, name: str):
    _dense(t, shape, torch.float32, name)
    return _ptr(t)


def _rows2(t: torch.Tensor, name: str):
    if t.dim() != 2:
        raise ValueError(f"expected {name} [T, C], got {tuple(t.shape)}")
    return t.shape


def _conv_args(x, w, bias, silu, T, C):
    a = _lib.SsmConvArgs()
    a.C, a.T_total, a.io, a.silu = C, T, _io(x, "x"), int(bool(silu))
    a.x, a.x_stride = x.data_ptr(), _rows(x, (T, C), x.dtype, "x")
    if w is None:
        raise ValueError("w is required")
    a.w, a.bias = _param(w, (C, 4), "w"), _param(bias, (C,), "bias")
    return a


def _packed(a, cu_dev, cu_host, check_cu_on_host: bool) -> int:
    a.N = cu_host.shape[0] - 1
    a.cu_seqlens = cu_dev.data_ptr()
    a.cu_seqlens_host = cu_host.ctypes.data if check_cu_on_host else None
    return a.N


def kda_ssm_conv(x: torch.Tensor, w: torch.Tensor, cu_seqlens, *, bias: Optional[torch.Tensor] = None,
                 silu: bool = True, conv_state_in: Optional[torch.Tensor] = None,
                 conv_state_out: Optional[torch.Tensor] = None, output_conv_state: bool = False,
                 y: Optional[torch.Tensor] = None, d_status=None, check_cu_on_host: bool = True, stream=None):
    """The selective scan's causal depthwise convolution of width 4 over packed sequences: x [T, C] (bf16 or fp32, rows
    may be strided), w [C, 4] fp32 (tap 3 multiplies x[t]), bias [C] fp32 or None; silu: SiLU after the sum.
    conv_state_in [N, C, 3] like x continues earlier tokens.  Returns y, or (y, conv_state_out [N, C, 3]) when
    output_conv_state is set or a conv_state_out is given."""
    lib = _lib.load()
    T, C = _rows2(x, "x")
    a = _conv_args(x, w, bias, silu, T, C)
    with _on(stream, x, w, bias, conv_state_in, conv_state_out, y, d_status) as s:
        cu_dev, cu_host = _cu_pair(cu_seqlens, x.device)
        N = _packed(a, cu_dev, cu_host, check_cu_on_host)
        _dense(conv_state_in, (N, C, 3), x.dtype, "conv_state_in")
        if y is None:
            y = torch.empty((T, C), dtype=x.dtype, device=x.device)
        if conv_state_out is None and output_conv_state:
            conv_state_out = torch.empty((N, C, 3), dtype=x.dtype, device=x.device)
        _dense(conv_state_out, (N, C, 3), x.dtype, "conv_state_out")
        _same_cuda_device(x=x, w=w, bias=bias, cu_seqlens=cu_dev, conv_state_in=conv_state_in,
                          conv_state_out=conv_state_out, y=y, d_status=d_status)
        a.conv_state_in, a.conv_state_out, a.d_status = _ptr(conv_state_in), _ptr(conv_state_out), _ptr(d_status)
        a.y, a.y_stride = y.data_ptr(), _rows(y, (T, C), x.dtype, "y")
        _check(lib.kda_ssm_conv(ctypes.byref(a), s), "kda_ssm_conv")
    return y if conv_state_out is None else (y, conv_state_out)


def kda_ssm_conv_step(x: torch.Tensor, w: torch.Tensor, conv_state: torch.Tensor, *,
                      bias: Optional[torch.Tensor] = None, silu: bool = True, y: Optional[torch.Tensor] = None,
                      stream=None) -> torch.Tensor:
    """One token for each of N sequences: x [N, C]; conv_state [N, C, 3] like x is rolled in place.  Returns y [N, C]."""
    lib = _lib.load()
    N, C = _rows2(x, "x")
    a = _conv_args(x, w, bias, silu, N, C)
    a.N = N
    if conv_state is None:
        raise ValueError("conv_state is required")
    _dense(conv_state, (N, C, 3), x.dtype, "conv_state")
    _same_cuda_device(x=x, w=w, bias=bias, conv_state=conv_state, y=y)
    with _on(stream, x, w, bias, conv_state, y) as s:
        if y is None:
            y = torch.empty((N, C), dtype=x.dtype, device=x.device)
        a.conv_state_out = conv_state.data_ptr()
        a.y, a.y_stride = y.data_ptr(), _rows(y, (N, C), x.dtype, "y")
        _check(lib.kda_ssm_conv_step(ctypes.byref(a), s), "kda_ssm_conv_step")
    return y


def kda_ssm_conv_backward(x: torch.Tensor, w: torch.Tensor, cu_seqlens, dy: torch.Tensor, *,
                          bias: Optional[torch.Tensor] = None, silu: bool = True,
                          conv_state_in: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                          d_status=None, check_cu_on_host: bool = True, stream=None) -> dict:
    """Gradients of sum(dy * y) of one kda_ssm_conv call (same inputs): a dict of dx (x's dtype), dw [C, 4] fp32, dbias
    [C] fp32 when bias is given, dconv_state_in [N, C, 3] fp32 when conv_state_in is given."""
    lib = _lib.load()
    T, C = _rows2(x, "x")
    b = _lib.SsmConvBackwardArgs()
    with _on(stream, x, w, bias, dy, conv_state_in, workspace, d_status) as s:
        cu_dev, cu_host = _cu_pair(cu_seqlens, x.device)
        b.fwd = _conv_args(x, w, bias, silu, T, C)
        N = _packed(b.fwd, cu_dev, cu_host, check_cu_on_host)
        _dense(conv_state_in, (N, C, 3), x.dtype, "conv_state_in")
        _same_cuda_device(x=x, w=w, bias=bias, dy=dy, cu_seqlens=cu_dev, conv_state_in=conv_state_in,
                          workspace=workspace, d_status=d_status)
        f32 = dict(dtype=torch.float32, device=x.device)
        res = {"dx": torch.empty((T, C), dtype=x.dtype, device=x.device), "dw": torch.empty((C, 4), **f32)}
        if bias is not None:
            res["dbias"] = torch.empty((C,), **f32)
        if conv_state_in is not None:
            res["dconv_state_in"] = torch.empty((N, C, 3), **f32)
        b.fwd.conv_state_in, b.fwd.d_status = _ptr(conv_state_in), _ptr(d_status)
        b.dy, b.dy_stride = dy.data_ptr(), _rows(dy, (T, C), x.dtype, "dy")
        b.dx, b.dw = res["dx"].data_ptr(), res["dw"].data_ptr()
        b.dbias, b.dconv_state_in = _ptr(res.get("dbias")), _ptr(res.get("dconv_state_in"))
        workspace = _workspace(lib.kda_ssm_conv_backward_workspace_size, b, "kda_ssm_conv_backward_workspace_size",
                               workspace, x.device)
        _check(lib.kda_ssm_conv_backward(ctypes.byref(b), s), "kda_ssm_conv_backward")
    return res


# ------------------------------------------------------------------ the selective scan
def _ssm_args(u, dt, A, B, C, *, D, z, dt_bias, softplus, rows, where):
    """SsmArgs with the inputs that prompt, step and gradients share, checked for shape and dtype."""
    if u.dim() != 2 or A.dim() != 2 or B.dim() != 3:
        raise ValueError(f"{where}: expected u [T, C], A [C, N] and B [T, G, N], got {tuple(u.shape)}, "
                         f"{tuple(A.shape)}, {tuple(B.shape)}")
    Ch, N, G = u.shape[1], A.shape[1], B.shape[1]
    a = _lib.SsmArgs()
    a.C, a.Nst, a.G, a.io, a.softplus = Ch, N, G, _io(u, "u"), int(bool(softplus))
    a.u, a.u_stride = u.data_ptr(), _rows(u, (rows, Ch), u.dtype, "u")
    a.dt, a.dt_stride = dt.data_ptr(), _rows(dt, (rows, Ch), u.dtype, "dt")
    a.A = _param(A, (Ch, N), "A")

    def grouped(t, name):
        if tuple(t.shape) != (rows, G, N) or t.dtype != u.dtype:
            raise ValueError(f"{name} must be {u.dtype} of shape {(rows, G, N)}, got {t.dtype} {tuple(t.shape)}")
        if (N > 1 and t.stride(2) != 1) or (G > 1 and t.stride(1) != N):
            raise ValueError(f"the (G, N) block of each row of {name} must be contiguous")
        return t.data_ptr(), (t.stride(0) if rows > 1 else G * N)

    a.B, a.B_stride = grouped(B, "B")
    a.Cm, a.C_stride = grouped(C, "C")
    a.D, a.dt_bias = _param(D, (Ch,), "D"), _param(dt_bias, (Ch,), "dt_bias")
    if z is not None:
        a.z, a.z_stride = z.data_ptr(), _rows(z, (rows, Ch), u.dtype, "z")
    return a, Ch, N, G


def kda_ssm_scan(u: torch.Tensor, dt: torch.Tensor, A: torch.Tensor, B: torch.Tensor, C: torch.Tensor, cu_seqlens, *,
                 D: Optional[torch.Tensor] = None, z: Optional[torch.Tensor] = None,
                 dt_bias: Optional[torch.Tensor] = None, softplus: bool = True,
                 initial_state: Optional[torch.Tensor] = None, output_final_state: bool = True,
                 final_state: Optional[torch.Tensor] = None, y: Optional[torch.Tensor] = None,
                 workspace: Optional[torch.Tensor] = None, d_status=None, check_cu_on_host: bool = True, stream=None):
    """The selective state space scan over packed sequences; returns (y, final_state or None).

    u, dt, z: [T, Ch] (bf16 or fp32, one dtype; rows may be strided); A [Ch, N] fp32 (<= 0; N in 8, 16, 32, 64);
    B, C: [T, G, N] like u, each group of Ch / G channels reads one; D, dt_bias [Ch] fp32 or None; z None: no gate.
    softplus: the step size is softplus(dt + dt_bias), else dt + dt_bias.  initial_state / final_state [num_sequences,
    Ch, N] fp32 (not the same buffer)."""
    lib = _lib.load()
    T = u.shape[0]
    a, Ch, N, G = _ssm_args(u, dt, A, B, C, D=D, z=z, dt_bias=dt_bias, softplus=softplus, rows=T, where="kda_ssm_scan")
    a.T_total = T
    with _on(stream, u, dt, A, B, C, D, z, dt_bias, initial_state, final_state, y, workspace, d_status) as s:
        cu_dev, cu_host = _cu_pair(cu_seqlens, u.device)
        n = _packed(a, cu_dev, cu_host, check_cu_on_host)
        if y is None:
            y = torch.empty((T, Ch), dtype=u.dtype, device=u.device)
        if final_state is None and output_final_state:
            final_state = torch.empty((n, Ch, N), dtype=torch.float32, device=u.device)
        a.initial_state = _param(initial_state, (n, Ch, N), "initial_state")
        a.final_state = _param(final_state, (n, Ch, N), "final_state")
        a.y, a.y_stride, a.d_status = y.data_ptr(), _rows(y, (T, Ch), u.dtype, "y"), _ptr(d_status)
        _same_cuda_device(u=u, dt=dt, A=A, B=B, C=C, D=D, z=z, dt_bias=dt_bias, cu_seqlens=cu_dev,
                          initial_state=initial_state, final_state=final_state, y=y, workspace=workspace,
                          d_status=d_status)
        workspace = _workspace(lib.kda_ssm_scan_workspace_size, a, "kda_ssm_scan_workspace_size", workspace, u.device)
        _check(lib.kda_ssm_scan(ctypes.byref(a), s), "kda_ssm_scan")
    return y, final_state


def kda_ssm_step(u: torch.Tensor, dt: torch.Tensor, A: torch.Tensor, B: torch.Tensor, C: torch.Tensor,
                 state: torch.Tensor, *, D: Optional[torch.Tensor] = None, z: Optional[torch.Tensor] = None,
                 dt_bias: Optional[torch.Tensor] = None, softplus: bool = True, y: Optional[torch.Tensor] = None,
                 stream=None) -> torch.Tensor:
    """One token for each of n sequences: u, dt, z [n, Ch], B, C [n, G, N]; state [n, Ch, N] fp32 is updated in place.
    Returns y [n, Ch]."""
    lib = _lib.load()
    n = u.shape[0]
    a, Ch, N, G = _ssm_args(u, dt, A, B, C, D=D, z=z, dt_bias=dt_bias, softplus=softplus, rows=n, where="kda_ssm_step")
    a.N = n
    if state is None:
        raise ValueError("state is required")
    a.final_state = _param(state, (n, Ch, N), "state")
    _same_cuda_device(u=u, dt=dt, A=A, B=B, C=C, state=state, D=D, z=z, dt_bias=dt_bias, y=y)
    with _on(stream, u, dt, A, B, C, state, D, z, dt_bias, y) as s:
        if y is None:
            y = torch.empty((n, Ch), dtype=u.dtype, device=u.device)
        a.y, a.y_stride = y.data_ptr(), _rows(y, (n, Ch), u.dtype, "y")
        _check(lib.kda_ssm_step(ctypes.byref(a), s), "kda_ssm_step")
    return y


def kda_ssm_backward(u: torch.Tensor, dt: torch.Tensor, A: torch.Tensor, B: torch.Tensor, C: torch.Tensor, cu_seqlens,
                     dy: torch.Tensor, *, D: Optional[torch.Tensor] = None, z: Optional[torch.Tensor] = None,
                     dt_bias: Optional[torch.Tensor] = None, softplus: bool = True,
                     initial_state: Optional[torch.Tensor] = None, d_final_state: Optional[torch.Tensor] = None,
                     workspace: Optional[torch.Tensor] = None, d_status=None, check_cu_on_host: bool = True,
                     stream=None) -> dict:
    """Gradients of sum(dy * y) + sum(d_final_state * final_state) of one kda_ssm_scan call (same inputs): a dict of du,
    ddt [T, Ch], dB, dC [T, G, N] (u's dtype), dA [Ch, N] fp32 and, where the input is given, dz (u's dtype), dD,
    ddt_bias [Ch] fp32 and dinitial_state fp32."""
    lib = _lib.load()
    T = u.shape[0]
    b = _lib.SsmBackwardArgs()
    f, Ch, N, G = _ssm_args(u, dt, A, B, C, D=D, z=z, dt_bias=dt_bias, softplus=softplus, rows=T,
                            where="kda_ssm_backward")
    f.T_total = T
    with _on(stream, u, dt, A, B, C, dy, D, z, dt_bias, initial_state, d_final_state, workspace, d_status) as s:
        cu_dev, cu_host = _cu_pair(cu_seqlens, u.device)
        n = _packed(f, cu_dev, cu_host, check_cu_on_host)
        f.initial_state = _param(initial_state, (n, Ch, N), "initial_state")
        f.d_status = _ptr(d_status)
        b.fwd = f
        b.dy, b.dy_stride = dy.data_ptr(), _rows(dy, (T, Ch), u.dtype, "dy")
        b.d_final_state = _param(d_final_state, (n, Ch, N), "d_final_state")
        _same_cuda_device(u=u, dt=dt, A=A, B=B, C=C, dy=dy, D=D, z=z, dt_bias=dt_bias, cu_seqlens=cu_dev,
                          initial_state=initial_state, d_final_state=d_final_state, workspace=workspace,
                          d_status=d_status)
        io, f32 = dict(dtype=u.dtype, device=u.device), dict(dtype=torch.float32, device=u.device)
        res = {"du": torch.empty((T, Ch), **io), "ddt": torch.empty((T, Ch), **io), "dA": torch.empty((Ch, N), **f32),
               "dB": torch.empty((T, G, N), **io), "dC": torch.empty((T, G, N), **io)}
        if z is not None:
            res["dz"] = torch.empty((T, Ch), **io)
        if D is not None:
            res["dD"] = torch.empty((Ch,), **f32)
        if dt_bias is not None:
            res["ddt_bias"] = torch.empty((Ch,), **f32)
        if initial_state is not None:
            res["dinitial_state"] = torch.empty((n, Ch, N), **f32)
        for name, t in res.items():
            setattr(b, name, t.data_ptr())
        workspace = _workspace(lib.kda_ssm_backward_workspace_size, b, "kda_ssm_backward_workspace_size", workspace,
                               u.device)
        _check(lib.kda_ssm_backward(ctypes.byref(b), s), "kda_ssm_backward")
    return res
