"""PyTorch-facing binding of the operators around the layer in a hybrid block: layer norm, 8-bit
storage of activations, and the selective state space scan with its short causal convolution.

Marshalling only, as in ``api``: the arithmetic runs in libkda.so.  Every tensor lives on the
current CUDA device.  Rows may be strided views (the last axis contiguous); outputs and workspace
are allocated on the stream that the call runs on.  Arguments travel as packed C structs
(``struct`` formats of the types in include/kda.h), since small calls are bound by this side.
"""
from __future__ import annotations

import contextlib
import ctypes
import struct
from typing import Optional

import numpy as np
import torch
from torch.autograd.function import once_differentiable

from . import _autograd, _lib
from .api import _DT, KDAError, _cu_pair

_F32, _U8 = torch.float32, torch.uint8
_BLOCK = _lib.KDA_PACK8_BLOCK

# the argument structs of include/kda.h, member by member ("0P" pads a struct that others follow)
_NORM = struct.Struct("@qii PqPPf PqP")
_NORM_BWD = struct.Struct("@qii PqPqP PPPq PPPN")
_CONV_FMT = "iiqii PP PqPP PPPqP 0P"
_CONV = struct.Struct("@" + _CONV_FMT)
_CONV_BWD = struct.Struct("@" + _CONV_FMT + "PqPq PPPPN")
_SSM_FMT = "iiiiqii PP PqPqP PqPqP PqPPP PqPNP 0P"
_SSM = struct.Struct("@" + _SSM_FMT)
_SSM_BWD = struct.Struct("@" + _SSM_FMT + "PqP PPPPPPPPPPN")


def _check(st: int, where: str) -> None:
    if st:
        raise KDAError(st, where)


@contextlib.contextmanager
def _on(stream, *inputs):
    """Makes `stream` current.  What the call allocates then belongs to it, and the inputs are marked as
    used on it, so that the allocator gives neither away before the kernels are done."""
    s = stream if isinstance(stream, torch.cuda.Stream) else torch.cuda.ExternalStream(int(stream))
    if s != torch.cuda.current_stream():
        for t in inputs:
            t = t[0] if isinstance(t, tuple) else t  # the device half of a cu_seqlens pair
            if isinstance(t, torch.Tensor) and t.is_cuda:
                t.record_stream(s)
    with torch.cuda.stream(s):
        yield


def _device(first: torch.Tensor, *others) -> int:
    """Index of the current device, on which every given tensor has to be: the library dereferences these
    pointers only on the GPU, and a host pointer there would fault."""
    index = first.get_device()
    for t in others:
        if t is not None and t.get_device() != index:
            raise ValueError(f"tensors are on {first.device} and on {t.device}; every tensor must be on one CUDA device")
    if index < 0:
        raise ValueError(f"tensors are on {first.device}; every tensor must be on a CUDA device")
    if index != torch._C._cuda_getDevice():  # CUDA is up: a tensor is on it
        raise ValueError(f"tensors are on {first.device} but the current device is cuda:{torch.cuda.current_device()}")
    return index


def _stream_of(index: int) -> int:
    return torch._C._cuda_getCurrentRawStream(index)


def _ptr(t: Optional[torch.Tensor]) -> int:
    return 0 if t is None else t.data_ptr()


def _status(t: Optional[torch.Tensor]) -> int:
    if t is None:
        return 0
    if t.dtype != torch.int32 or t.numel() < 1:
        raise ValueError(f"d_status must be an int32 tensor, got {t.dtype} {tuple(t.shape)}")
    return t.data_ptr()


def _io(t: torch.Tensor, name: str) -> int:
    io = _DT.get(t.dtype)
    if io is None:
        raise ValueError(f"{name} is {t.dtype}; expected bfloat16 or float32")
    return io


def _shape2(t: torch.Tensor, name: str):
    if t.dim() != 2:
        raise ValueError(f"expected {name} [rows, channels], got {tuple(t.shape)}")
    return t.shape


def _rows(t: torch.Tensor, M: int, C: int, dtype, name: str) -> int:
    """Row stride (elements) of a [M, C] tensor whose rows are dense."""
    if t.shape != (M, C):
        raise ValueError(f"{name} must be {(M, C)}, got {tuple(t.shape)}")
    if t.dtype != dtype:
        raise ValueError(f"{name} is {t.dtype}, expected {dtype}")
    s0, s1 = t.stride()
    if s1 != 1 and C > 1:
        raise ValueError(f"the rows of {name} must be contiguous")
    if M <= 1:
        return C
    if s0 < C:  # a broadcast row above all: to the library a stride of 0 means C
        raise ValueError(f"the rows of {name} overlap (stride {s0} below {C})")
    return s0


def _dense(t: Optional[torch.Tensor], shape, dtype, name: str) -> int:
    """Pointer of a contiguous tensor of this shape and dtype (0 for None)."""
    if t is None:
        return 0
    if t.shape != shape or t.dtype != dtype or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} tensor of shape {tuple(shape)}, "
                         f"got {t.dtype} {tuple(t.shape)}")
    return t.data_ptr()


_sizes: dict = {}  # workspace bytes by entry point, device and sizes: what the library answered


def _workspace(name: str, index: int, sizes, fmt, args, tail, workspace, device):
    """(pointer, bytes, tensor): the caller's buffer, or a new one of the size the library asks for.  The size is a
    function of the sizes and the device alone, so its answer is kept."""
    if workspace is None:
        key = (name, index, sizes)
        n = _sizes.get(key)
        if n is None:
            c = ctypes.c_size_t(0)
            _check(getattr(_lib.load(), name)(fmt.pack(*args, 0, 0, *tail), ctypes.byref(c)), name)
            if len(_sizes) >= 4096:
                _sizes.clear()
            n = _sizes[key] = c.value
        if n == 0:
            return 0, 0, None
        workspace = torch.empty(n, dtype=_U8, device=device)
        return workspace.data_ptr(), n, workspace
    if not workspace.is_contiguous():
        raise ValueError("workspace must be contiguous")
    return workspace.data_ptr(), workspace.numel() * workspace.element_size(), workspace


def _packed_cu(cu_seqlens, device):
    """(device int32 tensor, host int32 array, sequences).  A prepared pair is taken as it is."""
    if isinstance(cu_seqlens, tuple):
        dev, host = cu_seqlens
        if not (isinstance(host, np.ndarray) and host.dtype == np.int32 and host.flags.c_contiguous):
            host = np.ascontiguousarray(host, dtype=np.int32)
        if not isinstance(dev, torch.Tensor) or dev.dtype != torch.int32 or not dev.is_contiguous():
            raise ValueError("the device half of cu_seqlens must be a contiguous int32 tensor")
    else:
        dev, host = _cu_pair(cu_seqlens, device)
    if host.ndim != 1 or host.shape[0] < 1 or dev.numel() != host.shape[0]:
        raise ValueError("cu_seqlens must hold one more entry than there are sequences, on the device as on the host")
    return dev, host, host.shape[0] - 1


# ------------------------------------------------------------------ layer norm
def kda_layer_norm(x: torch.Tensor, weight: Optional[torch.Tensor] = None, bias: Optional[torch.Tensor] = None, *,
                   eps: float = 1e-5, y: Optional[torch.Tensor] = None, return_stats: bool = False, stream=None):
    """Layer norm over the last axis of x [M, C] (bf16 or fp32, rows may be strided); weight and bias [C] fp32 or
    None.  Returns y (x's dtype), or (y, stats) with return_stats: stats [M, 2] fp32 holds each row's mean and
    1 / sqrt(var + eps), which kda_layer_norm_backward reads.  C is at most 32768."""
    if stream is not None:
        with _on(stream, x, weight, bias, y):
            return kda_layer_norm(x, weight, bias, eps=eps, y=y, return_stats=return_stats)
    lib = _lib.load()
    M, C = _shape2(x, "x")
    io, dtype = _io(x, "x"), x.dtype
    xs, w, b = _rows(x, M, C, dtype, "x"), _dense(weight, (C,), _F32, "weight"), _dense(bias, (C,), _F32, "bias")
    ys = C if y is None else _rows(y, M, C, dtype, "y")
    index = _device(x, weight, bias, y)
    if y is None:
        y = torch.empty((M, C), dtype=dtype, device=x.device)
    stats = torch.empty((M, 2), dtype=_F32, device=x.device) if return_stats else None
    a = _NORM.pack(M, C, io, x.data_ptr(), xs, w, b, eps, y.data_ptr(), ys, _ptr(stats))
    _check(lib.kda_layer_norm(a, _stream_of(index)), "kda_layer_norm")
    return (y, stats) if return_stats else y


def kda_layer_norm_backward(dy: torch.Tensor, x: torch.Tensor, stats: torch.Tensor,
                            weight: Optional[torch.Tensor] = None, *, x_scales: Optional[torch.Tensor] = None,
                            param_grads: bool = True, workspace: Optional[torch.Tensor] = None, stream=None) -> dict:
    """Gradients of sum(dy * y) of one kda_layer_norm call: a dict of dx (dy's dtype) and, with param_grads, dweight
    and dbias [C] fp32 (summed in a fixed order).  x is the forward's input, or its 8-bit codes with x_scales given
    (the pair kda_pack8 returns), which the kernel reads directly; stats come from the forward."""
    if stream is not None:
        with _on(stream, dy, x, stats, weight, x_scales, workspace):
            return kda_layer_norm_backward(dy, x, stats, weight, x_scales=x_scales, param_grads=param_grads,
                                           workspace=workspace)
    lib = _lib.load()
    M, C = _shape2(dy, "dy")
    io, dtype, dev = _io(dy, "dy"), dy.dtype, dy.device
    dys = _rows(dy, M, C, dtype, "dy")
    if x_scales is None:
        xs, xp, sp = _rows(x, M, C, dtype, "x"), x.data_ptr(), 0
    else:
        xs, xp = C, _dense(x, (M, C), _U8, "x (8-bit codes)")
        sp = _dense(x_scales, (M, -(-C // _BLOCK)), _U8, "x_scales")
    st, w = _dense(stats, (M, 2), _F32, "stats"), _dense(weight, (C,), _F32, "weight")
    index = _device(dy, x, stats, weight, x_scales, workspace)
    res = {"dx": torch.empty((M, C), dtype=dtype, device=dev)}
    dw = db = 0
    if param_grads:
        res["dweight"] = gw = torch.empty((C,), dtype=_F32, device=dev)
        res["dbias"] = gb = torch.empty((C,), dtype=_F32, device=dev)
        dw, db = gw.data_ptr(), gb.data_ptr()
    args = (M, C, io, dy.data_ptr(), dys, xp, xs, sp, st, w, res["dx"].data_ptr(), C, dw, db)
    p, n, keep = 0, 0, None
    if param_grads:
        p, n, keep = _workspace("kda_layer_norm_backward_workspace_size", index, (M, C, io), _NORM_BWD, args, (),
                                workspace, dev)
    _check(lib.kda_layer_norm_backward(_NORM_BWD.pack(*args, p, n), _stream_of(index)), "kda_layer_norm_backward")
    return res


# ------------------------------------------------------------------ activations in 8 bits
def kda_pack8(x: torch.Tensor, *, stream=None):
    """x [M, C] (bf16 or fp32, rows may be strided) in 8 bits: (codes [M, C] uint8, scales [M, ceil(C / 32)] uint8).
    Each block of 32 channels is stored as e4m3 under the smallest power of two that keeps its largest magnitude
    within 448; scales hold the exponent + 127.  NaN and infinities come back as NaN."""
    if stream is not None:
        with _on(stream, x):
            return kda_pack8(x)
    lib = _lib.load()
    M, C = _shape2(x, "x")
    io, xs = _io(x, "x"), _rows(x, M, C, x.dtype, "x")
    index = _device(x)
    codes = torch.empty((M, C), dtype=_U8, device=x.device)
    scales = torch.empty((M, -(-C // _BLOCK)), dtype=_U8, device=x.device)
    _check(lib.kda_pack8(x.data_ptr(), xs, io, M, C, codes.data_ptr(), scales.data_ptr(), _stream_of(index)), "kda_pack8")
    return codes, scales


def kda_unpack8(codes: torch.Tensor, scales: torch.Tensor, *, dtype=torch.bfloat16, out: Optional[torch.Tensor] = None,
                stream=None) -> torch.Tensor:
    """The values that kda_pack8's codes and scales stand for, [M, C] in dtype (exact in bf16 and fp32 wherever the
    value itself is a normal number)."""
    if stream is not None:
        with _on(stream, codes, scales, out):
            return kda_unpack8(codes, scales, dtype=dtype, out=out)
    lib = _lib.load()
    M, C = _shape2(codes, "codes")
    cp, sp = _dense(codes, (M, C), _U8, "codes"), _dense(scales, (M, -(-C // _BLOCK)), _U8, "scales")
    if out is None and dtype not in _DT:
        raise ValueError(f"dtype is {dtype}; expected bfloat16 or float32")
    if out is not None:
        dtype = out.dtype
        _io(out, "out")
    xs = C if out is None else _rows(out, M, C, dtype, "out")
    index = _device(codes, scales, out)
    if out is None:
        out = torch.empty((M, C), dtype=dtype, device=codes.device)
    _check(lib.kda_unpack8(cp, sp, M, C, out.data_ptr(), xs, _DT[dtype], _stream_of(index)), "kda_unpack8")
    return out


# ------------------------------------------------------------------ the selective scan's short convolution
def _need(t, name: str):
    if t is None:
        raise ValueError(f"{name} is required")
    return t


def kda_ssm_conv(x: torch.Tensor, w: torch.Tensor, cu_seqlens, *, bias: Optional[torch.Tensor] = None,
                 silu: bool = True, conv_state_in: Optional[torch.Tensor] = None,
                 conv_state_out: Optional[torch.Tensor] = None, output_conv_state: bool = False,
                 y: Optional[torch.Tensor] = None, d_status=None, check_cu_on_host: bool = True, stream=None):
    """The selective scan's causal depthwise convolution of width 4 over packed sequences: x [T, C] (bf16 or fp32, rows
    may be strided), w [C, 4] fp32 (tap 3 multiplies x[t]), bias [C] fp32 or None; silu: SiLU after the sum.
    conv_state_in [N, C, 3] like x continues earlier tokens.  Returns y, or (y, conv_state_out [N, C, 3]) when
    output_conv_state is set or a conv_state_out is given."""
    if stream is not None:
        with _on(stream, x, w, cu_seqlens, bias, conv_state_in, conv_state_out, y, d_status):
            return kda_ssm_conv(x, w, cu_seqlens, bias=bias, silu=silu, conv_state_in=conv_state_in,
                                conv_state_out=conv_state_out, output_conv_state=output_conv_state, y=y,
                                d_status=d_status, check_cu_on_host=check_cu_on_host)
    lib = _lib.load()
    T, C = _shape2(x, "x")
    io, dtype, dev = _io(x, "x"), x.dtype, x.device
    xs, wp, bp = _rows(x, T, C, dtype, "x"), _dense(_need(w, "w"), (C, 4), _F32, "w"), _dense(bias, (C,), _F32, "bias")
    ys = C if y is None else _rows(y, T, C, dtype, "y")
    cu, host, N = _packed_cu(cu_seqlens, dev)
    index = _device(x, w, cu, bias, conv_state_in, conv_state_out, y, d_status)
    if conv_state_out is None and output_conv_state:
        conv_state_out = torch.empty((N, C, 3), dtype=dtype, device=dev)
    si = _dense(conv_state_in, (N, C, 3), dtype, "conv_state_in")
    so = _dense(conv_state_out, (N, C, 3), dtype, "conv_state_out")
    if y is None:
        y = torch.empty((T, C), dtype=dtype, device=dev)
    a = _CONV.pack(N, C, T, io, bool(silu), cu.data_ptr(), host.ctypes.data if check_cu_on_host else 0, x.data_ptr(), xs,
                   wp, bp, si, so, y.data_ptr(), ys, _status(d_status))
    _check(lib.kda_ssm_conv(a, _stream_of(index)), "kda_ssm_conv")
    return y if conv_state_out is None else (y, conv_state_out)


def kda_ssm_conv_step(x: torch.Tensor, w: torch.Tensor, conv_state: torch.Tensor, *,
                      bias: Optional[torch.Tensor] = None, silu: bool = True, y: Optional[torch.Tensor] = None,
                      stream=None) -> torch.Tensor:
    """One token for each of N sequences: x [N, C]; conv_state [N, C, 3] like x is rolled in place.  Returns y [N, C]."""
    if stream is not None:
        with _on(stream, x, w, conv_state, bias, y):
            return kda_ssm_conv_step(x, w, conv_state, bias=bias, silu=silu, y=y)
    lib = _lib.load()
    N, C = _shape2(x, "x")
    io, dtype = _io(x, "x"), x.dtype
    xs, wp, bp = _rows(x, N, C, dtype, "x"), _dense(_need(w, "w"), (C, 4), _F32, "w"), _dense(bias, (C,), _F32, "bias")
    sp = _dense(_need(conv_state, "conv_state"), (N, C, 3), dtype, "conv_state")
    ys = C if y is None else _rows(y, N, C, dtype, "y")
    index = _device(x, w, conv_state, bias, y)
    if y is None:
        y = torch.empty((N, C), dtype=dtype, device=x.device)
    a = _CONV.pack(N, C, 0, io, bool(silu), 0, 0, x.data_ptr(), xs, wp, bp, 0, sp, y.data_ptr(), ys, 0)
    _check(lib.kda_ssm_conv_step(a, _stream_of(index)), "kda_ssm_conv_step")
    return y


def kda_ssm_conv_backward(x: torch.Tensor, w: torch.Tensor, cu_seqlens, dy: torch.Tensor, *,
                          bias: Optional[torch.Tensor] = None, silu: bool = True,
                          conv_state_in: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                          d_status=None, check_cu_on_host: bool = True, stream=None) -> dict:
    """Gradients of sum(dy * y) of one kda_ssm_conv call (same inputs): a dict of dx (x's dtype), dw [C, 4] fp32, dbias
    [C] fp32 when bias is given, dconv_state_in [N, C, 3] fp32 when conv_state_in is given."""
    if stream is not None:
        with _on(stream, x, w, cu_seqlens, dy, bias, conv_state_in, workspace, d_status):
            return kda_ssm_conv_backward(x, w, cu_seqlens, dy, bias=bias, silu=silu, conv_state_in=conv_state_in,
                                         workspace=workspace, d_status=d_status, check_cu_on_host=check_cu_on_host)
    lib = _lib.load()
    T, C = _shape2(x, "x")
    io, dtype, dev = _io(x, "x"), x.dtype, x.device
    xs, wp, bp = _rows(x, T, C, dtype, "x"), _dense(_need(w, "w"), (C, 4), _F32, "w"), _dense(bias, (C,), _F32, "bias")
    dys = _rows(dy, T, C, dtype, "dy")
    cu, host, N = _packed_cu(cu_seqlens, dev)
    index = _device(x, w, cu, dy, bias, conv_state_in, workspace, d_status)
    si = _dense(conv_state_in, (N, C, 3), dtype, "conv_state_in")
    res = {"dx": torch.empty((T, C), dtype=dtype, device=dev), "dw": torch.empty((C, 4), dtype=_F32, device=dev)}
    if bias is not None:
        res["dbias"] = torch.empty((C,), dtype=_F32, device=dev)
    if conv_state_in is not None:
        res["dconv_state_in"] = torch.empty((N, C, 3), dtype=_F32, device=dev)
    args = (N, C, T, io, bool(silu), cu.data_ptr(), host.ctypes.data if check_cu_on_host else 0, x.data_ptr(), xs, wp, bp,
            si, 0, 0, 0, _status(d_status), dy.data_ptr(), dys, res["dx"].data_ptr(), C, res["dw"].data_ptr(),
            _ptr(res.get("dbias")), _ptr(res.get("dconv_state_in")))
    p, n, keep = _workspace("kda_ssm_conv_backward_workspace_size", index, (T, C, io), _CONV_BWD, args, (), workspace, dev)
    _check(lib.kda_ssm_conv_backward(_CONV_BWD.pack(*args, p, n), _stream_of(index)), "kda_ssm_conv_backward")
    return res


# ------------------------------------------------------------------ the selective scan
def _grouped(t: torch.Tensor, rows: int, G: int, N: int, dtype, name: str) -> int:
    """Row stride of a [rows, G, N] tensor whose (G, N) block is dense."""
    if t.dim() != 3 or t.shape != (rows, G, N) or t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype} of shape {(rows, G, N)}, got {t.dtype} {tuple(t.shape)}")
    s0, s1, s2 = t.stride()
    if (N > 1 and s2 != 1) or (G > 1 and s1 != N):
        raise ValueError(f"the (G, N) block of each row of {name} must be contiguous")
    if rows <= 1:
        return G * N
    if s0 < G * N:
        raise ValueError(f"the rows of {name} overlap (stride {s0} below {G * N})")
    return s0


def _ssm_inputs(u, dt, A, B, C, D, z, dt_bias):
    """Checked shapes, dtypes and strides of the inputs that prompt, step and gradients share: the sizes, and the
    values of kda_ssm_args from u to dt_bias."""
    if u.dim() != 2 or A.dim() != 2 or B.dim() != 3:
        raise ValueError(f"expected u [T, C], A [C, N] and B [T, G, N], got {tuple(u.shape)}, {tuple(A.shape)}, "
                         f"{tuple(B.shape)}")
    T, Ch = u.shape
    N, G, dtype = A.shape[1], B.shape[1], u.dtype
    io = _io(u, "u")
    vals = (u.data_ptr(), _rows(u, T, Ch, dtype, "u"), dt.data_ptr(), _rows(dt, T, Ch, dtype, "dt"),
            _dense(A, (Ch, N), _F32, "A"), B.data_ptr(), _grouped(B, T, G, N, dtype, "B"), C.data_ptr(),
            _grouped(C, T, G, N, dtype, "C"), _dense(D, (Ch,), _F32, "D"), _ptr(z),
            0 if z is None else _rows(z, T, Ch, dtype, "z"), _dense(dt_bias, (Ch,), _F32, "dt_bias"))
    return T, Ch, N, G, io, dtype, vals


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
    if stream is not None:
        with _on(stream, u, dt, A, B, C, cu_seqlens, D, z, dt_bias, initial_state, final_state, y, workspace, d_status):
            return kda_ssm_scan(u, dt, A, B, C, cu_seqlens, D=D, z=z, dt_bias=dt_bias, softplus=softplus,
                                initial_state=initial_state, output_final_state=output_final_state,
                                final_state=final_state, y=y, workspace=workspace, d_status=d_status,
                                check_cu_on_host=check_cu_on_host)
    lib = _lib.load()
    T, Ch, N, G, io, dtype, vals = _ssm_inputs(u, dt, A, B, C, D, z, dt_bias)
    ys, dev = Ch if y is None else _rows(y, T, Ch, dtype, "y"), u.device
    cu, host, n = _packed_cu(cu_seqlens, dev)
    index = _device(u, dt, A, B, C, cu, D, z, dt_bias, initial_state, final_state, y, workspace, d_status)
    ip = _dense(initial_state, (n, Ch, N), _F32, "initial_state")
    if final_state is None and output_final_state:
        final_state = torch.empty((n, Ch, N), dtype=_F32, device=dev)
    fp = _dense(final_state, (n, Ch, N), _F32, "final_state")
    if y is None:
        y = torch.empty((T, Ch), dtype=dtype, device=dev)
    args = (n, Ch, N, G, T, io, bool(softplus), cu.data_ptr(), host.ctypes.data if check_cu_on_host else 0, *vals, ip, fp,
            y.data_ptr(), ys)
    status = _status(d_status)
    p, size, keep = _workspace("kda_ssm_scan_workspace_size", index, (T, Ch, N, G, io), _SSM, args, (status,), workspace, dev)
    _check(lib.kda_ssm_scan(_SSM.pack(*args, p, size, status), _stream_of(index)), "kda_ssm_scan")
    return y, final_state


def kda_ssm_step(u: torch.Tensor, dt: torch.Tensor, A: torch.Tensor, B: torch.Tensor, C: torch.Tensor,
                 state: torch.Tensor, *, D: Optional[torch.Tensor] = None, z: Optional[torch.Tensor] = None,
                 dt_bias: Optional[torch.Tensor] = None, softplus: bool = True, y: Optional[torch.Tensor] = None,
                 stream=None) -> torch.Tensor:
    """One token for each of n sequences: u, dt, z [n, Ch], B, C [n, G, N]; state [n, Ch, N] fp32 is updated in place.
    Returns y [n, Ch]."""
    if stream is not None:
        with _on(stream, u, dt, A, B, C, state, D, z, dt_bias, y):
            return kda_ssm_step(u, dt, A, B, C, state, D=D, z=z, dt_bias=dt_bias, softplus=softplus, y=y)
    lib = _lib.load()
    n, Ch, N, G, io, dtype, vals = _ssm_inputs(u, dt, A, B, C, D, z, dt_bias)
    sp = _dense(_need(state, "state"), (n, Ch, N), _F32, "state")
    ys = Ch if y is None else _rows(y, n, Ch, dtype, "y")
    index = _device(u, dt, A, B, C, state, D, z, dt_bias, y)
    if y is None:
        y = torch.empty((n, Ch), dtype=dtype, device=u.device)
    a = _SSM.pack(n, Ch, N, G, 0, io, bool(softplus), 0, 0, *vals, 0, sp, y.data_ptr(), ys, 0, 0, 0)
    _check(lib.kda_ssm_step(a, _stream_of(index)), "kda_ssm_step")
    return y


def kda_ssm_backward(u: torch.Tensor, dt: torch.Tensor, A: torch.Tensor, B: torch.Tensor, C: torch.Tensor, cu_seqlens,
                     dy: torch.Tensor, *, D: Optional[torch.Tensor] = None, z: Optional[torch.Tensor] = None,
                     dt_bias: Optional[torch.Tensor] = None, softplus: bool = True,
                     initial_state: Optional[torch.Tensor] = None, d_final_state: Optional[torch.Tensor] = None,
                     workspace: Optional[torch.Tensor] = None, d_status=None, check_cu_on_host: bool = True,
                     stream=None) -> dict:
    """Gradients of sum(dy * y) + sum(d_final_state * final_state) of one kda_ssm_scan call (same inputs): a dict of du,
    ddt [T, Ch], dB, dC [T, G, N] (u's dtype), dA [Ch, N] fp32 and, where the input is given, dz (u's dtype), dD,
    ddt_bias [Ch] fp32 and dinitial_state fp32.  The workspace holds the states in front of every fourth token:
    about T * Ch * N bytes."""
    if stream is not None:
        with _on(stream, u, dt, A, B, C, cu_seqlens, dy, D, z, dt_bias, initial_state, d_final_state, workspace, d_status):
            return kda_ssm_backward(u, dt, A, B, C, cu_seqlens, dy, D=D, z=z, dt_bias=dt_bias, softplus=softplus,
                                    initial_state=initial_state, d_final_state=d_final_state, workspace=workspace,
                                    d_status=d_status, check_cu_on_host=check_cu_on_host)
    lib = _lib.load()
    T, Ch, N, G, io, dtype, vals = _ssm_inputs(u, dt, A, B, C, D, z, dt_bias)
    dys, dev = _rows(dy, T, Ch, dtype, "dy"), u.device
    cu, host, n = _packed_cu(cu_seqlens, dev)
    index = _device(u, dt, A, B, C, cu, dy, D, z, dt_bias, initial_state, d_final_state, workspace, d_status)
    ip = _dense(initial_state, (n, Ch, N), _F32, "initial_state")
    dfp = _dense(d_final_state, (n, Ch, N), _F32, "d_final_state")

    def io_rows(*shape):
        return torch.empty(shape, dtype=dtype, device=dev)

    def params(*shape):
        return torch.empty(shape, dtype=_F32, device=dev)

    res = {"du": io_rows(T, Ch), "ddt": io_rows(T, Ch), "dA": params(Ch, N), "dB": io_rows(T, G, N), "dC": io_rows(T, G, N)}
    if z is not None:
        res["dz"] = io_rows(T, Ch)
    if D is not None:
        res["dD"] = params(Ch)
    if dt_bias is not None:
        res["ddt_bias"] = params(Ch)
    if initial_state is not None:
        res["dinitial_state"] = params(n, Ch, N)
    args = (n, Ch, N, G, T, io, bool(softplus), cu.data_ptr(), host.ctypes.data if check_cu_on_host else 0, *vals, ip, 0,
            0, 0, 0, 0, _status(d_status), dy.data_ptr(), dys, dfp,
            *(_ptr(res.get(k)) for k in ("du", "ddt", "dA", "dB", "dC", "dD", "dz", "ddt_bias", "dinitial_state")))
    p, size, keep = _workspace("kda_ssm_backward_workspace_size", index, (T, Ch, N, G, io), _SSM_BWD, args, (), workspace, dev)
    _check(lib.kda_ssm_backward(_SSM_BWD.pack(*args, p, size), _stream_of(index)), "kda_ssm_backward")
    return res


# ------------------------------------------------------------------ differentiable forms
def _keep(t: Optional[torch.Tensor], saved: str):
    """(t, None), or t [M, C] as 8-bit codes and scales."""
    return (t, None) if t is None or saved == "io" else kda_pack8(t)


def _restore(t: Optional[torch.Tensor], scales: Optional[torch.Tensor], dtype):
    return t if scales is None else kda_unpack8(t, scales, dtype=dtype)


class _NormLayer(torch.autograd.Function):
    """kda_layer_norm forward, kda_layer_norm_backward backward."""

    @staticmethod
    def forward(ctx, x, weight, bias, eps, saved):
        y, stats = kda_layer_norm(x, weight, bias, eps=eps, return_stats=True)
        if any(ctx.needs_input_grad):
            ctx.save_for_backward(*_keep(x, saved), stats, weight)
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
    mean and deviation.  In a captured graph, see kda_ssm_layer's note."""
    _autograd.check_saved(saved)
    return _autograd.apply(_NormLayer, "kda_norm_layer", x, weight, bias, float(eps), saved)


class _SsmConvLayer(torch.autograd.Function):
    """kda_ssm_conv forward, kda_ssm_conv_backward backward."""

    @staticmethod
    def forward(ctx, x, w, bias, conv_state_in, cu_pair, silu, saved):
        y = kda_ssm_conv(x, w, cu_pair, bias=bias, silu=silu, conv_state_in=conv_state_in)
        if any(ctx.needs_input_grad):
            ctx.save_for_backward(*_keep(x, saved), w, bias, conv_state_in)
            ctx.rest = (cu_pair, silu, x.dtype)
        return y

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        x, scales, w, bias, state = ctx.saved_tensors
        cu_pair, silu, dtype = ctx.rest
        g = kda_ssm_conv_backward(_restore(x, scales, dtype), w, cu_pair, dy.contiguous(), bias=bias, silu=silu,
                                  conv_state_in=state)
        want = ctx.needs_input_grad
        dstate = g["dconv_state_in"].to(state.dtype) if want[3] else None
        return (g["dx"] if want[0] else None, g["dw"] if want[1] else None, g["dbias"] if want[2] else None, dstate,
                None, None, None)


def kda_ssm_conv_layer(x: torch.Tensor, w: torch.Tensor, cu_seqlens, *, bias: Optional[torch.Tensor] = None,
                       silu: bool = True, conv_state_in: Optional[torch.Tensor] = None, saved: str = "io") -> torch.Tensor:
    """kda_ssm_conv as a differentiable PyTorch operation: y, with gradients for x, w, bias and conv_state_in.
    saved="e4m3" keeps x in 8 bits for the backward pass.  In a captured graph, see kda_ssm_layer's note."""
    _autograd.check_saved(saved)
    return _autograd.apply(_SsmConvLayer, "kda_ssm_conv_layer", x, w, bias, conv_state_in,
                           _cu_pair(cu_seqlens, x.device), bool(silu), saved)


class _SsmLayer(torch.autograd.Function):
    """kda_ssm_scan forward, kda_ssm_backward backward."""

    @staticmethod
    def forward(ctx, u, dt, A, B, C, D, z, dt_bias, initial_state, cu_pair, softplus, saved):
        y, fin = kda_ssm_scan(u, dt, A, B, C, cu_pair, D=D, z=z, dt_bias=dt_bias, softplus=softplus,
                              initial_state=initial_state)
        if any(ctx.needs_input_grad):
            ctx.save_for_backward(*_keep(u, saved), *_keep(z, saved), dt, A, B, C, D, dt_bias, initial_state)
            ctx.rest = (cu_pair, softplus, u.dtype)
        ctx.set_materialize_grads(False)
        return y, fin

    @staticmethod
    @once_differentiable
    def backward(ctx, dy, dfin):
        u, us, z, zs, dt, A, B, C, D, dt_bias, init = ctx.saved_tensors
        cu_pair, softplus, dtype = ctx.rest
        dy = torch.zeros(dt.shape, dtype=dtype, device=dt.device) if dy is None else dy.contiguous()
        g = kda_ssm_backward(_restore(u, us, dtype), dt, A, B, C, cu_pair, dy, D=D, z=_restore(z, zs, dtype),
                             dt_bias=dt_bias, softplus=softplus, initial_state=init,
                             d_final_state=None if dfin is None else dfin.contiguous())
        names = ("du", "ddt", "dA", "dB", "dC", "dD", "dz", "ddt_bias", "dinitial_state")
        return (*(g[n] if want else None for n, want in zip(names, ctx.needs_input_grad)), None, None, None)


def kda_ssm_layer(u: torch.Tensor, dt: torch.Tensor, A: torch.Tensor, B: torch.Tensor, C: torch.Tensor, cu_seqlens, *,
                  D: Optional[torch.Tensor] = None, z: Optional[torch.Tensor] = None,
                  dt_bias: Optional[torch.Tensor] = None, softplus: bool = True,
                  initial_state: Optional[torch.Tensor] = None, saved: str = "io"):
    """kda_ssm_scan as a differentiable PyTorch operation: (y, final_state), with gradients for u, dt, A, B, C, D, z,
    dt_bias and initial_state.  saved="e4m3" keeps u and z in 8 bits for the backward pass; dt, B and C stay as they
    are (a step size enters the decays' exponents, and B and C are small).

    In a captured graph: pass cu_seqlens as a prepared (device, host) pair, and let no eager graph of the same leaves,
    built on the default stream, live; the call raises if one that it knows of does (a forward pass that is captured
    alone runs under torch.no_grad())."""
    _autograd.check_saved(saved)
    return _autograd.apply(_SsmLayer, "kda_ssm_layer", u, dt, A, B, C, D, z, dt_bias, initial_state,
                           _cu_pair(cu_seqlens, u.device), bool(softplus), saved)
