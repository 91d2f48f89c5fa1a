"""PyTorch-facing binding of a decode step over few tokens: weights stored in 4 bits and their projections, a
mixture-of-experts layer, and the verification of drafted tokens.

Marshalling only, as in ``block``: the arithmetic runs in libkda.so.  Nothing here has a gradient; weights in 4 bits
are codes, and a choice of tokens or experts is discrete.
"""
from __future__ import annotations

import struct
from typing import Optional, Tuple, Union

import torch

from . import _lib
from .api import _DT, _EPI
from .block import (_F32, _U8, _check, _dense, _device, _io, _on, _packed_cu, _ptr, _rows, _shape2, _status, _stream_of,
                    _workspace)

_BF16 = torch.bfloat16
_FORMAT = {"e2m1": _lib.KDA_WEIGHT_E2M1, "int4": _lib.KDA_WEIGHT_INT4}
_SCORE = {"sigmoid": _lib.KDA_SCORE_SIGMOID, "softmax": _lib.KDA_SCORE_SOFTMAX}

# the argument structs of include/kda.h, member by member
_PACK4 = struct.Struct("@qiPqiiiiPP")
_GEMM4 = struct.Struct("@iiiPqiiiPPPqii PNP")
_MOE = struct.Struct("@iiiiiPqPiPifiiiPPPPPqiPP PNP")
_VERIFY = struct.Struct("@iqiiPqPqPiPPPPPP")

Weight = Union[torch.Tensor, Tuple[torch.Tensor, torch.Tensor]]


# format and type of scales by the scales' dtype
_SCALES = {_U8: (_lib.KDA_WEIGHT_E2M1, 0), **{d: (_lib.KDA_WEIGHT_INT4, v) for d, v in _DT.items()}}


def _weight4(codes: torch.Tensor, scales: torch.Tensor, name: str):
    """(format, group, scale dtype, K) of 4-bit weights [..., K / 2] with scales [..., K / group]."""
    kind, cs, ss = _SCALES.get(scales.dtype), codes.shape, scales.shape
    if kind is None:
        raise ValueError(f"the scales of {name} are {scales.dtype}; expected uint8 (e2m1), bfloat16 or float32 (int4)")
    if codes.dtype is not _U8 or len(cs) < 2 or not codes.is_contiguous():
        raise ValueError(f"the codes of {name} must be a contiguous uint8 tensor [..., rows, K / 2], got {codes.dtype} {tuple(cs)}")
    if ss[:-1] != cs[:-1] or not scales.is_contiguous():
        raise ValueError(f"the scales of {name} must be contiguous, one row of them per row of codes {tuple(cs)}, got {tuple(ss)}")
    K, groups = 2 * cs[-1], ss[-1]
    if groups < 1 or K % groups:
        raise ValueError(f"{groups} scales do not divide the {K} weights of a row of {name}")
    return kind[0], K // groups, kind[1], K


def kda_pack4(w: torch.Tensor, *, format: str = "e2m1", group: int = 32, scale_dtype=torch.bfloat16, stream=None):
    """Weights w [..., rows, K] (bf16 or fp32) in 4 bits: (codes [..., rows, K / 2] uint8, scales [..., rows, K / group]).
    Two codes share a byte, the even k in its low half.  format "e2m1": 32 weights under the smallest power of two that
    keeps their largest magnitude within 6, scales uint8 (exponent + 127, as kda_pack8's).  format "int4": codes hold
    round(w / scale) + 8, scale = max|w| / 7 in scale_dtype (bf16 or fp32), group 32, 64 or 128.  w must be finite."""
    if stream is not None:
        with _on(stream, w):
            return kda_pack4(w, format=format, group=group, scale_dtype=scale_dtype)
    if w.dim() < 2:
        raise ValueError(f"expected w [..., rows, K], got {tuple(w.shape)}")
    if format not in _FORMAT:
        raise ValueError(f"format is {format!r}; expected 'e2m1' or 'int4'")
    if format == "int4" and scale_dtype not in _DT:
        raise ValueError(f"scale_dtype is {scale_dtype}; expected bfloat16 or float32")
    *lead, K = w.shape
    if group < 1 or K < 1 or K % group:
        raise ValueError(f"K = {K} is not a multiple of the group of {group}")
    flat = w if w.dim() == 2 else w.reshape(-1, K)
    rows, io = flat.shape[0], _io(w, "w")
    ws = _rows(flat, rows, K, w.dtype, "w")
    index = _device(w)
    codes = torch.empty((*lead, K // 2), dtype=_U8, device=w.device)
    sdt = _U8 if format == "e2m1" else scale_dtype
    scales = torch.empty((*lead, K // group), dtype=sdt, device=w.device)
    a = _PACK4.pack(rows, K, flat.data_ptr(), ws, io, _FORMAT[format], group, _DT.get(sdt, 0), codes.data_ptr(), scales.data_ptr())
    _check(_lib.load().kda_pack4(a, _stream_of(index)), "kda_pack4")
    return codes, scales


def kda_unpack4(codes: torch.Tensor, scales: torch.Tensor, *, dtype=torch.bfloat16, stream=None) -> torch.Tensor:
    """The weights [..., rows, K] (bf16 or fp32) that 4-bit codes and scales stand for; the format is told by the scales'
    type (uint8: e2m1)."""
    if stream is not None:
        with _on(stream, codes, scales):
            return kda_unpack4(codes, scales, dtype=dtype)
    fmt, group, sdt, K = _weight4(codes, scales, "w")
    if dtype not in _DT:
        raise ValueError(f"dtype is {dtype}; expected bfloat16 or float32")
    index = _device(codes, scales)
    w = torch.empty((*codes.shape[:-1], K), dtype=dtype, device=codes.device)
    a = _PACK4.pack(w.numel() // K if K else 0, K, w.data_ptr(), K, _DT[dtype], fmt, group, sdt, codes.data_ptr(), scales.data_ptr())
    _check(_lib.load().kda_unpack4(a, _stream_of(index)), "kda_unpack4")
    return w


def kda_gemm4(A: torch.Tensor, codes: torch.Tensor, scales: torch.Tensor, *, epilogue: str = "none",
              out: Optional[torch.Tensor] = None, out_dtype=None, workspace: Optional[torch.Tensor] = None, d_status=None,
              stream=None) -> torch.Tensor:
    """C = epilogue(A @ W^T) for the few rows of a decode step: A [M, K] bf16 (rows may be strided), W [N, K] in 4 bits
    (codes [N, K / 2] and scales [N, K / group] as kda_pack4 returns them).  Epilogues and out_dtype as in kda_gemm; out
    [M, N] may have strided rows.  Sums are fp32, in a fixed order, rounded once (e2m1, more than 96 rows, bf16 result: cut off, by
    an eighth of that rounding at most).  e2m1 up to 96 rows, or with an fp32 result: what lies below 2^-22 of the largest of 32
    values of A is dropped.  Integer codes are for few rows: from some 32 on kda_gemm on bf16 weights is faster.  M is at
    most 65535."""
    if stream is not None:
        with _on(stream, A, codes, scales, out, workspace, d_status):
            return kda_gemm4(A, codes, scales, epilogue=epilogue, out=out, out_dtype=out_dtype, workspace=workspace,
                             d_status=d_status)
    M, K = _shape2(A, "A")
    if codes.dim() != 2:
        raise ValueError(f"expected codes [N, K / 2], got {tuple(codes.shape)}")
    fmt, group, sdt, Kw = _weight4(codes, scales, "W")
    if Kw != K:
        raise ValueError(f"A has {K} columns, W {Kw}")
    epi = _EPI.get(epilogue)
    if epi is None:
        raise ValueError(f"epilogue is {epilogue!r}; expected one of {tuple(_EPI)}")
    N, lda = codes.shape[0], _rows(A, M, K, _BF16, "A")
    index = _device(A, codes, scales, out, workspace, d_status)
    dev = A.device
    if out is None:
        dt = out_dtype or (_BF16 if epi == _lib.KDA_EPI_NONE else _F32)
        if dt not in _DT:
            raise ValueError(f"out_dtype is {dt}; expected bfloat16 or float32")
        out, ldc = torch.empty((M, N), dtype=dt, device=dev), N
    else:
        if out_dtype is not None and out.dtype != out_dtype:
            raise ValueError(f"out is {out.dtype}, out_dtype {out_dtype}")
        _io(out, "out")
        ldc = _rows(out, M, N, out.dtype, "out")
    args = (M, N, K, A.data_ptr(), lda, fmt, group, sdt, codes.data_ptr(), scales.data_ptr(), out.data_ptr(), ldc,
            _DT[out.dtype], epi)
    st = 0 if d_status is None else _status(d_status)
    p, n, keep = _workspace("kda_gemm4_workspace_size", index, (M, N, K, fmt, group), _GEMM4, args, (st,), workspace, dev)
    _check(_lib.load().kda_gemm4(_GEMM4.pack(*args, p, n, st), _stream_of(index)), "kda_gemm4")
    return out


def _experts(w: Weight, rows: int, E: int, K: int, name: str):
    """(format, group, scale dtype, codes or weights, scales or None) of the experts' weights [E, rows, K]."""
    if isinstance(w, torch.Tensor):
        _dense(w, (E, rows, K), _BF16, name)
        return _lib.KDA_WEIGHT_BF16, 0, 0, w, None
    codes, scales = w
    fmt, group, sdt, Kw = _weight4(codes, scales, name)
    if codes.shape != (E, rows, K // 2) or Kw != K:
        raise ValueError(f"{name} must be {(E, rows, K)}, got {(*codes.shape[:-1], Kw)}")
    return fmt, group, sdt, codes, scales


def kda_moe(x: torch.Tensor, router: torch.Tensor, w_in: Weight, w_out: Weight, top: int, *,
            bias: Optional[torch.Tensor] = None, score: str = "sigmoid", scale: float = 1.0,
            y: Optional[torch.Tensor] = None, out_dtype=None, return_routing: bool = False,
            workspace: Optional[torch.Tensor] = None, d_status=None, stream=None):
    """A mixture-of-experts layer for few tokens: x [M, D] bf16 (rows may be strided), router [E, D] bf16 or fp32.
    Each token takes the `top` experts with the largest score + bias (score "sigmoid" of its logits; bias [E] fp32 or
    None) or the largest logits ("softmax"), ties to the lower expert, weighted by their scores divided by the sum of
    the chosen ones, times `scale`; an expert computes W_out (silu(g) u) with g and u the halves of W_in x.  w_in
    [E, 2 F, D] and w_out [E, D, F] are bf16 tensors or (codes, scales) in one 4-bit format (kda_pack4).  Returns y
    [M, D] in out_dtype (default bf16), or (y, ids [M, top] int32, weights [M, top] fp32), best first, with
    return_routing.  A token whose logits are not finite gets NaN.  M * top is at most 65535, E 1024, top 32; made for the tokens of
    a decode step, slow for a prompt's (an expert's weights pass again for every few of its tokens)."""
    if stream is not None:
        pair = lambda w: (w,) if isinstance(w, torch.Tensor) else w  # noqa: E731
        with _on(stream, x, router, *pair(w_in), *pair(w_out), bias, y, workspace, d_status):
            return kda_moe(x, router, w_in, w_out, top, bias=bias, score=score, scale=scale, y=y, out_dtype=out_dtype,
                           return_routing=return_routing, workspace=workspace, d_status=d_status)
    lib = _lib.load()
    M, D = _shape2(x, "x")
    E, _ = _shape2(router, "router")
    mode = _SCORE.get(score)
    if mode is None:
        raise ValueError(f"score is {score!r}; expected one of {tuple(_SCORE)}")
    first = w_in if isinstance(w_in, torch.Tensor) else w_in[0]
    if first.dim() != 3 or first.shape[1] % 2:
        raise ValueError(f"expected w_in [E, 2 F, D], got {tuple(first.shape)}")
    F = first.shape[1] // 2
    fmt, group, sdt, wi, si = _experts(w_in, 2 * F, E, D, "w_in")
    fmt2, group2, sdt2, wo, so = _experts(w_out, D, E, F, "w_out")
    if (fmt, group, sdt) != (fmt2, group2, sdt2):
        raise ValueError("w_in and w_out must be in one format, with one group and one type of scales")
    xs = _rows(x, M, D, _BF16, "x")
    rdt = _io(router, "router")
    r = _dense(router, (E, D), router.dtype, "router")
    b = _dense(bias, (E,), _F32, "bias")
    index = _device(x, router, wi, si, wo, so, bias, y, workspace, d_status)
    dev = x.device
    if y is None:
        dt = out_dtype or _BF16
        if dt not in _DT:
            raise ValueError(f"out_dtype is {dt}; expected bfloat16 or float32")
        y, ys = torch.empty((M, D), dtype=dt, device=dev), D
    else:
        if out_dtype is not None and y.dtype != out_dtype:
            raise ValueError(f"y is {y.dtype}, out_dtype {out_dtype}")
        _io(y, "y")
        ys = _rows(y, M, D, y.dtype, "y")
    ids = weights = None
    ip = wp = 0
    if return_routing and top > 0:
        ids, weights = torch.empty((M, top), dtype=torch.int32, device=dev), torch.empty((M, top), dtype=_F32, device=dev)
        ip, wp = ids.data_ptr(), weights.data_ptr()
    args = (M, E, top, D, F, x.data_ptr(), xs, r, rdt, b, mode, scale, fmt, group, sdt, wi.data_ptr(), _ptr(si), wo.data_ptr(),
            _ptr(so), y.data_ptr(), ys, _DT[y.dtype], ip, wp)
    st = 0 if d_status is None else _status(d_status)
    p, n, keep = _workspace("kda_moe_workspace_size", index, (M, E, top, D, F, fmt, group, b != 0), _MOE, args, (st,),
                            workspace, dev)
    _check(lib.kda_moe(_MOE.pack(*args, p, n, st), _stream_of(index)), "kda_moe")
    return (y, ids, weights) if return_routing else y


def kda_verify(target: torch.Tensor, tokens: torch.Tensor, u: torch.Tensor, cu_seqlens, *,
               draft: Optional[torch.Tensor] = None, d_status=None, check_cu_on_host: bool = True, stream=None):
    """Which drafted tokens stand.  Rows are packed as the multi-token decode runs them: a sequence of L drafts has
    L + 1 rows.  target [T, V] (bf16 or fp32): the target's probabilities after each row; draft [T, V] (same type): what
    the drafts were drawn from, None for a drafter that proposes its best token; tokens [T] int32 or int64: row i holds
    the draft after it; u [T] fp32 in [0, 1).  The last row of a sequence has no draft.  A draft d is taken while
    u draft(d) < target(d); after the first refusal, or after all, one token is drawn by the last row's u from
    max(target - draft, 0), or from the last row's target.  Values not above 0, NaN among them, count as 0; an infinity in what
    is drawn from, or a sum beyond fp32, draws -1, as a row of zeros does.  Returns (tokens [T]: the accepted drafts, the drawn token,
    then -1; accepted [N] int32)."""
    if stream is not None:
        with _on(stream, target, tokens, u, cu_seqlens, draft, d_status):
            return kda_verify(target, tokens, u, cu_seqlens, draft=draft, d_status=d_status, check_cu_on_host=check_cu_on_host)
    lib = _lib.load()
    T, V = _shape2(target, "target")
    io = _io(target, "target")
    ps = _rows(target, T, V, target.dtype, "target")
    qs = V if draft is None else _rows(draft, T, V, target.dtype, "draft")
    if tokens.dtype not in (torch.int32, torch.int64):
        raise ValueError(f"tokens are {tokens.dtype}; expected int32 or int64")
    d, up = _dense(tokens, (T,), tokens.dtype, "tokens"), _dense(u, (T,), _F32, "u")
    cu_dev, cu_host, N = _packed_cu(cu_seqlens, target.device)
    index = _device(target, tokens, u, cu_dev, draft, d_status)
    out = torch.empty((T,), dtype=tokens.dtype, device=target.device)
    accepted = torch.empty((N,), dtype=torch.int32, device=target.device)
    a = _VERIFY.pack(N, T, V, io, target.data_ptr(), ps, _ptr(draft), qs, d, tokens.element_size(), up, cu_dev.data_ptr(),
                     cu_host.ctypes.data if check_cu_on_host else 0, out.data_ptr(), accepted.data_ptr(), _status(d_status))
    _check(lib.kda_verify(a, _stream_of(index)), "kda_verify")
    return out, accepted
