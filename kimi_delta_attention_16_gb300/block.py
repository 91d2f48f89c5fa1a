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
from .api import _DT, KDAError, _same_cuda_device

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
