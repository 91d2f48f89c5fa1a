"""Host-side checks of 4-bit weights, the mixture of experts and the verification of drafts: refused with a status before
anything is launched.  No GPU is needed, and no pointer is dereferenced on the host."""
import ctypes

import numpy as np
import pytest
import torch

import kimi_delta_attention_16_gb300 as kda
from kimi_delta_attention_16_gb300 import _lib, serve

BASE, STEP = 0x7f0000000000, 0x400000000
INVALID, UNSUPPORTED, WORKSPACE = _lib.KDA_ERR_INVALID_ARG, _lib.KDA_ERR_UNSUPPORTED, _lib.KDA_ERR_WORKSPACE


def at(i, off=0):
    return BASE + i * STEP + off


def call(name, a):
    st = getattr(_lib.load(), name)(ctypes.byref(a), None)
    if st:
        assert _lib.load().kda_last_error()
    return st


def fill(a, kw):
    for k, v in kw.items():
        setattr(a, k, v)
    return a


def test_structs_match_the_binding():
    """The packed formats lay every member of the C structs where their mirrors have it."""
    for fmt, cls in ((serve._PACK4, _lib.Pack4Args), (serve._GEMM4, _lib.Gemm4Args), (serve._MOE, _lib.MoeArgs),
                     (serve._VERIFY, _lib.VerifyArgs)):
        values = [0.5 if t is ctypes.c_float else 1000 + i for i, (_, t) in enumerate(cls._fields_)]
        got = cls.from_buffer_copy(fmt.pack(*values))
        assert fmt.size == ctypes.sizeof(cls)
        for (name, _), v in zip(cls._fields_, values):
            assert getattr(got, name) == v, name


def pack4(**kw):
    a = _lib.Pack4Args()
    a.rows, a.K, a.w, a.w_dtype, a.format, a.group = 4, 128, at(0), _lib.KDA_BF16, _lib.KDA_WEIGHT_E2M1, 32
    a.codes, a.scales = at(1), at(2)
    return fill(a, kw)


INT4 = dict(format=_lib.KDA_WEIGHT_INT4)


@pytest.mark.parametrize("kw,code", [
    (dict(rows=-1), INVALID), (dict(K=0), INVALID), (dict(K=48), UNSUPPORTED), (dict(K=(1 << 28) + 32), UNSUPPORTED),
    (dict(w_dtype=2), INVALID), (dict(format=0), INVALID), (dict(format=3), INVALID), (dict(group=64), UNSUPPORTED),
    (dict(INT4, group=16), UNSUPPORTED), (dict(INT4, group=128, K=192), UNSUPPORTED), (dict(INT4, scale_dtype=5), INVALID),
    (dict(w=None), INVALID), (dict(codes=None), INVALID), (dict(scales=None), INVALID), (dict(w=at(0, 1)), INVALID),
    (dict(w_stride=127), INVALID), (dict(codes=at(1, 8)), INVALID), (dict(INT4, scales=at(2, 1)), INVALID),
    (dict(codes=at(0, 16)), INVALID), (dict(scales=at(1, 255)), INVALID), (dict(w_stride=1 << 58), UNSUPPORTED)])
def test_pack4_refusals(kw, code):
    assert call("kda_pack4", pack4(**kw)) == code
    assert call("kda_unpack4", pack4(**kw)) == code


def gemm4(**kw):
    a = _lib.Gemm4Args()
    a.M, a.N, a.K, a.A, a.lda, a.format, a.group = 4, 100, 256, at(0), 256, _lib.KDA_WEIGHT_E2M1, 32
    a.codes, a.scales, a.C, a.ldc, a.c_dtype = at(1), at(2), at(3), 100, _lib.KDA_BF16
    a.workspace, a.workspace_bytes = at(4), 1 << 24
    return fill(a, kw)


@pytest.mark.parametrize("kw,code", [
    (dict(M=-1), INVALID), (dict(N=-1), INVALID), (dict(K=0), INVALID), (dict(K=40), UNSUPPORTED),
    (dict(M=65536), UNSUPPORTED), (dict(N=(1 << 24) + 1), UNSUPPORTED), (dict(K=(1 << 24) + 32, lda=1 << 25), UNSUPPORTED),
    (dict(format=_lib.KDA_WEIGHT_BF16), INVALID), (dict(group=128), UNSUPPORTED), (dict(INT4, scale_dtype=2), INVALID),
    (dict(c_dtype=7), INVALID), (dict(epilogue=3), INVALID), (dict(epilogue=-1), INVALID), (dict(A=None), INVALID),
    (dict(A=at(0, 1)), INVALID), (dict(lda=255), INVALID), (dict(ldc=99), INVALID), (dict(C=None), INVALID),
    (dict(C=at(0)), INVALID), (dict(C=at(1, 128)), INVALID), (dict(C=at(2, 2)), INVALID), (dict(codes=at(1, 4)), INVALID),
    (dict(codes=None), INVALID), (dict(scales=None), INVALID), (dict(lda=1 << 58), UNSUPPORTED), (dict(workspace=None), WORKSPACE),
    (dict(workspace_bytes=4096), WORKSPACE), (dict(workspace=at(4, 16)), WORKSPACE), (dict(workspace=at(1)), INVALID),
    (dict(workspace=at(3)), INVALID)])
def test_gemm4_refusals(kw, code):
    assert call("kda_gemm4", gemm4(**kw)) == code


def moe(**kw):
    a = _lib.MoeArgs()
    a.M, a.E, a.top, a.D, a.F, a.x, a.router, a.scale = 4, 16, 2, 256, 128, at(0), at(1), 1.0
    a.format, a.group = _lib.KDA_WEIGHT_E2M1, 32
    a.bias, a.w_in, a.w_in_scales, a.w_out, a.w_out_scales, a.y, a.ids, a.weights = (at(i) for i in range(2, 10))
    a.workspace, a.workspace_bytes = at(10), 1 << 24
    return fill(a, kw)


@pytest.mark.parametrize("kw,code", [
    (dict(M=-1), INVALID), (dict(E=0), INVALID), (dict(D=0), INVALID), (dict(F=0), INVALID), (dict(top=0), INVALID),
    (dict(top=17), INVALID), (dict(E=1025), UNSUPPORTED), (dict(E=64, top=33), UNSUPPORTED), (dict(M=40000), UNSUPPORTED),
    (dict(D=(1 << 20) + 32), UNSUPPORTED), (dict(E=1024, F=1 << 20), UNSUPPORTED), (dict(D=250), UNSUPPORTED), (dict(F=100), UNSUPPORTED), (dict(format=0, F=100), UNSUPPORTED),
    (dict(router_dtype=3), INVALID), (dict(y_dtype=3), INVALID), (dict(score=2), INVALID), (dict(score=1), INVALID),
    (dict(x=None), INVALID), (dict(y=None), INVALID), (dict(router=None), INVALID), (dict(w_in=None), INVALID),
    (dict(w_out=at(5, 8)), INVALID), (dict(w_in_scales=None), INVALID), (dict(x_stride=100), INVALID), (dict(y=at(0)), INVALID),
    (dict(y=at(3)), INVALID), (dict(ids=at(9)), INVALID), (dict(bias=at(2, 2)), INVALID), (dict(ids=at(8, 1)), INVALID),
    (dict(workspace=None), WORKSPACE), (dict(workspace_bytes=100), WORKSPACE), (dict(workspace=at(10, 16)), WORKSPACE),
    (dict(workspace=at(5)), INVALID), (dict(workspace=at(7)), INVALID)])
def test_moe_refusals(kw, code):
    assert call("kda_moe", moe(**kw)) == code


def test_moe_workspace_size():
    n = ctypes.c_size_t(1)
    assert _lib.load().kda_moe_workspace_size(ctypes.byref(moe()), ctypes.byref(n)) == 0
    assert n.value >= 4 * 16 * 16 + 8 * (128 + 256) * 4 and n.value % 256 == 0
    assert _lib.load().kda_moe_workspace_size(ctypes.byref(moe(M=0)), ctypes.byref(n)) == 0 and n.value == 0
    assert _lib.load().kda_moe_workspace_size(ctypes.byref(moe(top=0)), ctypes.byref(n)) == INVALID


def test_gemm4_workspace_size():
    n = ctypes.c_size_t(1)
    size = _lib.load().kda_gemm4_workspace_size
    assert size(ctypes.byref(gemm4()), ctypes.byref(n)) == 0 and n.value >= 4 * 256 * 4
    assert size(ctypes.byref(gemm4(**INT4)), ctypes.byref(n)) == 0 and n.value >= 4 * 256 * 2
    assert size(ctypes.byref(gemm4(N=0)), ctypes.byref(n)) == 0 and n.value == 0
    assert size(ctypes.byref(gemm4(K=7)), ctypes.byref(n)) == UNSUPPORTED


def verify(**kw):
    a = _lib.VerifyArgs()
    a.N, a.T_total, a.V, a.dtype, a.target, a.draft, a.tokens, a.token_bytes = 2, 6, 100, _lib.KDA_FP32, at(0), at(1), at(2), 4
    a.u, a.cu_seqlens, a.out, a.accepted = at(3), at(4), at(5), at(6)
    cu = np.array(kw.pop("cu", [0, 2, 6]), np.int32)
    a.cu_seqlens_host = cu.ctypes.data
    a._keep = cu
    return fill(a, kw)


@pytest.mark.parametrize("kw,code", [
    (dict(N=-1), INVALID), (dict(T_total=-1), INVALID), (dict(V=0), INVALID), (dict(V=4000001), UNSUPPORTED),
    (dict(T_total=1 << 31), UNSUPPORTED), (dict(dtype=2), INVALID), (dict(token_bytes=2), INVALID), (dict(cu_seqlens=None), INVALID),
    (dict(cu=[0, 2, 5]), INVALID), (dict(cu=[0, 7, 6]), INVALID), (dict(cu=[1, 2, 6]), INVALID), (dict(N=0, cu=[6]), INVALID),
    (dict(accepted=None), INVALID), (dict(accepted=at(6, 2)), INVALID), (dict(target=None), INVALID), (dict(target=at(0, 2)), INVALID),
    (dict(target_stride=99), INVALID), (dict(draft_stride=50), INVALID), (dict(tokens=None), INVALID), (dict(u=None), INVALID),
    (dict(out=None), INVALID), (dict(out=at(2)), INVALID), (dict(out=at(6)), INVALID), (dict(accepted=at(4, 8)), INVALID),
    (dict(token_bytes=8, tokens=at(2, 4)), INVALID)])
def test_verify_refusals(kw, code):
    assert call("kda_verify", verify(**kw)) == code


def test_empty_calls_launch_nothing():
    assert call("kda_pack4", pack4(rows=0)) == 0
    assert call("kda_gemm4", gemm4(M=0, A=None)) == 0
    assert call("kda_gemm4", gemm4(N=0, C=None)) == 0
    assert call("kda_moe", moe(M=0, x=None)) == 0
    a = verify(N=0, T_total=0, cu=[0])
    assert call("kda_verify", a) == 0
    for name in ("kda_pack4", "kda_unpack4", "kda_gemm4", "kda_moe", "kda_verify"):
        assert getattr(_lib.load(), name)(None, None) == INVALID


def test_binding_refusals():
    """What the binding turns away before the library sees it."""
    bf, u8 = torch.bfloat16, torch.uint8
    x = torch.zeros(2, 64, dtype=bf)
    codes, scales = torch.zeros(5, 32, dtype=u8), torch.zeros(5, 2, dtype=u8)
    bad = [lambda: kda.kda_gemm4(x, codes, scales),  # not on a GPU
           lambda: kda.kda_gemm4(x.float(), codes, scales), lambda: kda.kda_gemm4(x[0], codes, scales),
           lambda: kda.kda_gemm4(x, codes[:, :16], scales), lambda: kda.kda_gemm4(x, codes.int(), scales),
           lambda: kda.kda_gemm4(x, codes, scales[:3]), lambda: kda.kda_gemm4(x, codes, scales.half()),
           lambda: kda.kda_gemm4(x, codes, torch.zeros(5, 3, dtype=u8)), lambda: kda.kda_gemm4(x, codes, scales, epilogue="relu"),
           lambda: kda.kda_gemm4(x[:1].expand(4, 64), codes, scales),
           lambda: kda.kda_pack4(x, format="fp4"), lambda: kda.kda_pack4(x, group=48), lambda: kda.kda_pack4(x[0]),
           lambda: kda.kda_pack4(x, format="int4", scale_dtype=torch.float16), lambda: kda.kda_unpack4(codes, scales, dtype=torch.half),
           lambda: kda.kda_verify(torch.zeros(3, 9), torch.zeros(3), torch.zeros(3), [0, 3]),
           lambda: kda.kda_verify(torch.zeros(3, 9), torch.zeros(2, dtype=torch.int32), torch.zeros(3), [0, 3]),
           lambda: kda.kda_verify(torch.zeros(3, 9), torch.zeros(3, dtype=torch.int32), torch.zeros(3), [0, 3], draft=torch.zeros(3, 9, dtype=bf))]
    r, wi, wo = torch.zeros(4, 64, dtype=bf), torch.zeros(4, 64, 64, dtype=bf), torch.zeros(4, 64, 32, dtype=bf)
    q = lambda w: (torch.zeros(*w.shape[:-1], w.shape[-1] // 2, dtype=u8), torch.zeros(*w.shape[:-1], w.shape[-1] // 32, dtype=u8))  # noqa: E731
    bad += [lambda: kda.kda_moe(x, r, wi, wo, 2), lambda: kda.kda_moe(x, r, q(wi), wo, 2), lambda: kda.kda_moe(x, r, wi, wo, 2, score="max"),
            lambda: kda.kda_moe(x, r, wi[:, :63], wo, 2), lambda: kda.kda_moe(x, r, wi, wo[:3], 2), lambda: kda.kda_moe(x, r.half(), wi, wo, 2),
            lambda: kda.kda_moe(x, r, wi, wo, 2, bias=torch.zeros(3))]
    for f in bad:
        with pytest.raises((ValueError, kda.KDAError)):
            f()
