"""Host-side checks of the operators around the layer: sizes, dtypes, pointers, strides, overlaps and workspaces are
refused with a status before anything is launched.  No GPU is needed, and no pointer is dereferenced on the host."""
import ctypes

import numpy as np
import pytest
import torch

import kimi_delta_attention_16_gb300 as kda
from kimi_delta_attention_16_gb300 import _lib

BASE = 0x7f0000000000
STEP = 0x40000000  # between the made-up buffers
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
        obj, _, field = k.rpartition("__")
        setattr(getattr(a, obj) if obj else a, field, v)
    return a


def norm(**kw):
    a = _lib.NormArgs()
    a.M, a.C, a.io, a.eps = 4, 100, _lib.KDA_BF16, 1e-5
    a.x, a.weight, a.bias, a.y, a.stats = at(0), at(1), at(2), at(3), at(4)
    return fill(a, kw)


@pytest.mark.parametrize("kw,code", [
    (dict(M=-1), INVALID), (dict(C=0), INVALID), (dict(C=32769), UNSUPPORTED), (dict(io=2), INVALID),
    (dict(x=None), INVALID), (dict(y=None), INVALID), (dict(x=at(0, 1)), INVALID), (dict(x_stride=99), INVALID),
    (dict(y_stride=-100), INVALID), (dict(weight=at(1, 2)), INVALID), (dict(y=at(0)), INVALID),
    (dict(y=at(0, 700)), INVALID), (dict(stats=at(3, 8)), INVALID), (dict(stats=at(4, 4)), INVALID), (dict(y=at(1)), INVALID),
    (dict(x_stride=1 << 58, M=4), UNSUPPORTED)])
def test_layer_norm_refusals(kw, code):
    assert call("kda_layer_norm", norm(**kw)) == code


def norm_bwd(**kw):
    a = _lib.NormBackwardArgs()
    a.M, a.C, a.io = 4, 100, _lib.KDA_BF16
    a.dy, a.x, a.stats, a.weight, a.dx, a.dweight, a.dbias = (at(i) for i in range(7))
    a.workspace, a.workspace_bytes = at(8), 1 << 30
    return fill(a, kw)


@pytest.mark.parametrize("kw,code", [
    (dict(M=-1), INVALID), (dict(C=40000), UNSUPPORTED), (dict(dy=None), INVALID), (dict(x=None), INVALID),
    (dict(stats=None), INVALID), (dict(stats=at(2, 4)), INVALID), (dict(dx=None), INVALID), (dict(dx=at(0)), INVALID), (dict(dweight=at(6)), INVALID),
    (dict(workspace=None), WORKSPACE), (dict(workspace_bytes=16), WORKSPACE), (dict(workspace=at(8, 16)), WORKSPACE),
    (dict(workspace=at(2)), INVALID), (dict(x_scales=at(4)), INVALID), (dict(dy_stride=10), INVALID)])
def test_layer_norm_backward_refusals(kw, code):
    assert call("kda_layer_norm_backward", norm_bwd(**kw)) == code


@pytest.mark.parametrize("M,C,dtype,x,stride,codes,scales,code", [
    (-1, 8, 0, at(0), 0, at(1), at(2), INVALID), (4, 0, 0, at(0), 0, at(1), at(2), INVALID),
    (4, 8, 3, at(0), 0, at(1), at(2), INVALID), (4, 8, 0, None, 0, at(1), at(2), INVALID),
    (4, 8, 0, at(0), 0, None, at(2), INVALID), (4, 8, 0, at(0), 7, at(1), at(2), INVALID),
    (4, 8, 1, at(0, 2), 0, at(1), at(2), INVALID), (4, 8, 0, at(0), 0, at(0, 8), at(2), INVALID),
    (4, 8, 0, at(0), 0, at(1), at(1, 31), INVALID), (1, (1 << 30) + 1, 0, at(0), 0, at(40), at(80), UNSUPPORTED)])
def test_pack8_refusals(M, C, dtype, x, stride, codes, scales, code):
    lib = _lib.load()
    assert lib.kda_pack8(x, stride, dtype, M, C, codes, scales, None) == code
    assert lib.kda_unpack8(codes, scales, M, C, x, stride, dtype, None) == code


CU = np.array([0, 10, 24], np.int32)


def conv(**kw):
    a = _lib.SsmConvArgs()
    a.N, a.C, a.T_total, a.io, a.silu = 2, 48, 24, _lib.KDA_BF16, 1
    a.cu_seqlens, a.cu_seqlens_host = at(0), CU.ctypes.data
    a.x, a.w, a.bias, a.conv_state_in, a.conv_state_out, a.y = (at(i) for i in range(1, 7))
    return fill(a, kw)


BAD_CU = np.array([0, 30, 24], np.int32)
CONV_BAD = [(dict(N=-1), INVALID), (dict(C=0), INVALID), (dict(C=(1 << 20) + 1), UNSUPPORTED), (dict(io=5), INVALID),
            (dict(T_total=25), INVALID), (dict(cu_seqlens=None), INVALID), (dict(cu_seqlens_host=BAD_CU.ctypes.data), INVALID),
            (dict(x=None), INVALID), (dict(w=None), INVALID), (dict(x_stride=47), INVALID), (dict(x=at(1, 1)), INVALID),
            (dict(bias=at(3, 1)), INVALID), (dict(conv_state_in=at(4, 1)), INVALID),
            (dict(T_total=1 << 31, cu_seqlens_host=None), UNSUPPORTED)]


@pytest.mark.parametrize("kw,code", CONV_BAD + [
    (dict(y=None), INVALID), (dict(y=at(1)), INVALID), (dict(conv_state_out=at(4, 16)), INVALID), (dict(y=at(2)), INVALID)])
def test_ssm_conv_refusals(kw, code):
    assert call("kda_ssm_conv", conv(**kw)) == code


@pytest.mark.parametrize("kw,code", [
    (dict(conv_state_out=None), INVALID), (dict(conv_state_in=at(9)), INVALID), (dict(N=-2), INVALID), (dict(y=at(1)), INVALID),
    (dict(x=None), INVALID), (dict(w=None), INVALID), (dict(io=-1), INVALID)])
def test_ssm_conv_step_refusals(kw, code):
    assert call("kda_ssm_conv_step", conv(**{"conv_state_in": None, **kw})) == code


def conv_bwd(**kw):
    a = _lib.SsmConvBackwardArgs()
    a.fwd = conv(conv_state_out=None, y=None)
    a.dy, a.dx, a.dw, a.dbias, a.dconv_state_in = (at(i) for i in range(10, 15))
    a.workspace, a.workspace_bytes = at(20), 1 << 30
    return fill(a, kw)


@pytest.mark.parametrize("kw,code", [({"fwd__" + k: v for k, v in kw.items()}, c) for kw, c in CONV_BAD] + [
    (dict(dy=None), INVALID), (dict(dx=None), INVALID), (dict(dw=None), INVALID), (dict(dx=at(10)), INVALID),
    (dict(dx=at(1)), INVALID), (dict(dw=at(13)), INVALID), (dict(workspace=None), WORKSPACE),
    (dict(workspace_bytes=1), WORKSPACE), (dict(workspace=at(12)), INVALID), (dict(dconv_state_in=at(14, 2)), INVALID)])
def test_ssm_conv_backward_refusals(kw, code):
    assert call("kda_ssm_conv_backward", conv_bwd(**kw)) == code


def ssm(**kw):
    a = _lib.SsmArgs()
    a.N, a.C, a.Nst, a.G, a.T_total, a.io, a.softplus = 2, 48, 16, 2, 24, _lib.KDA_BF16, 1
    a.cu_seqlens, a.cu_seqlens_host = at(0), CU.ctypes.data
    a.u, a.dt, a.A, a.B, a.Cm, a.D, a.z, a.dt_bias, a.initial_state, a.final_state, a.y = (at(i) for i in range(1, 12))
    a.workspace, a.workspace_bytes = at(30), 1 << 30
    return fill(a, kw)


SSM_BAD = [(dict(N=-1), INVALID), (dict(C=0), INVALID), (dict(Nst=12), UNSUPPORTED), (dict(Nst=128), UNSUPPORTED),
           (dict(G=0), INVALID), (dict(G=5), INVALID), (dict(io=9), INVALID), (dict(T_total=23), INVALID),
           (dict(cu_seqlens=None), INVALID), (dict(u=None), INVALID), (dict(dt=None), INVALID), (dict(A=None), INVALID),
           (dict(B=None), INVALID), (dict(Cm=None), INVALID), (dict(u_stride=40), INVALID), (dict(B_stride=31), INVALID),
           (dict(z=at(7, 1)), INVALID), (dict(A=at(3, 8)), INVALID), (dict(D=at(6, 2)), INVALID),
           (dict(initial_state=at(9, 4)), INVALID), (dict(C=1 << 21, G=1), UNSUPPORTED)]


@pytest.mark.parametrize("kw,code", SSM_BAD + [
    (dict(y=None), INVALID), (dict(y=at(1)), INVALID), (dict(y=at(4, 2)), INVALID), (dict(final_state=at(9)), INVALID),
    (dict(final_state=at(9, 64)), INVALID), (dict(final_state=at(10, 4)), INVALID), (dict(y=at(10)), INVALID)])
def test_ssm_scan_refusals(kw, code):
    assert call("kda_ssm_scan", ssm(**kw)) == code


@pytest.mark.parametrize("kw,code", [
    (dict(initial_state=at(9)), INVALID), (dict(final_state=None), INVALID), (dict(Nst=4), UNSUPPORTED), (dict(G=7), INVALID),
    (dict(u=None), INVALID), (dict(y=at(10)), INVALID), (dict(N=-1), INVALID), (dict(io=2), INVALID), (dict(A=None), INVALID),
    (dict(u_stride=1 << 31), UNSUPPORTED), (dict(B_stride=1 << 32), UNSUPPORTED)])
def test_ssm_step_refusals(kw, code):
    assert call("kda_ssm_step", ssm(**{"initial_state": None, **kw})) == code


def ssm_bwd(**kw):
    a = _lib.SsmBackwardArgs()
    a.fwd = ssm(final_state=None, y=None)
    (a.dy, a.d_final_state, a.du, a.ddt, a.dA, a.dB, a.dC, a.dD, a.dz, a.ddt_bias,
     a.dinitial_state) = (at(i) for i in range(12, 23))
    a.workspace, a.workspace_bytes = at(40), 1 << 30
    return fill(a, kw)


@pytest.mark.parametrize("kw,code", [({"fwd__" + k: v for k, v in kw.items()}, c) for kw, c in SSM_BAD] + [
    (dict(dy=None), INVALID), (dict(du=None), INVALID), (dict(ddt=None), INVALID), (dict(dA=None), INVALID),
    (dict(dB=None), INVALID), (dict(dC=None), INVALID), (dict(fwd__z=None), INVALID), (dict(du=at(12)), INVALID),
    (dict(du=at(1)), INVALID), (dict(ddt=at(14)), INVALID), (dict(dinitial_state=at(13)), INVALID),
    (dict(dinitial_state=at(22, 8)), INVALID), (dict(workspace=None), WORKSPACE), (dict(workspace_bytes=4096), WORKSPACE),
    (dict(workspace=at(40, 128)), WORKSPACE), (dict(workspace=at(16)), INVALID), (dict(dy_stride=-48), INVALID)])
def test_ssm_backward_refusals(kw, code):
    assert call("kda_ssm_backward", ssm_bwd(**kw)) == code


def test_nothing_to_do_launches_nothing():
    """No rows or no sequences: accepted without a device."""
    zero = np.zeros(1, np.int32)
    assert call("kda_layer_norm", norm(M=0, x=None, y=None)) == 0
    assert _lib.load().kda_pack8(None, 0, 0, 0, 8, None, None, None) == 0
    assert call("kda_ssm_conv", conv(N=0, T_total=0, cu_seqlens=None, cu_seqlens_host=zero.ctypes.data)) == 0
    assert call("kda_ssm_scan", ssm(N=0, T_total=0, cu_seqlens=None, cu_seqlens_host=None)) == 0
    assert call("kda_ssm_step", ssm(N=0, initial_state=None)) == 0
    assert call("kda_ssm_conv_step", conv(N=0)) == 0


def test_workspace_sizes():
    """Sizes grow with the problem, fit what the call then asks for, and NULL answers are refused."""
    lib, n = _lib.load(), ctypes.c_size_t(7)
    for name, a in (("kda_layer_norm_backward", norm_bwd()), ("kda_ssm_conv_backward", conv_bwd()), ("kda_ssm_scan", ssm()),
                    ("kda_ssm_backward", ssm_bwd())):
        f = getattr(lib, name + "_workspace_size")
        assert f(ctypes.byref(a), None) == INVALID and f(None, ctypes.byref(n)) == INVALID and n.value == 0
        assert f(ctypes.byref(a), ctypes.byref(n)) == 0
    a = ssm_bwd()
    a.fwd.T_total = 4096
    assert lib.kda_ssm_backward_workspace_size(ctypes.byref(a), ctypes.byref(n)) == 0
    assert n.value >= 4096 // 4 * 48 * 16 * 4
    small = norm_bwd(dweight=None, dbias=None)
    assert lib.kda_layer_norm_backward_workspace_size(ctypes.byref(small), ctypes.byref(n)) == 0 and n.value == 0


def test_binding_refusals():
    """The Python entry points refuse wrong shapes, dtypes, strides and host tensors."""
    x, w = torch.zeros(4, 8), torch.ones(8)
    codes, scales = torch.zeros(4, 8, dtype=torch.uint8), torch.zeros(4, 1, dtype=torch.uint8)
    st = torch.zeros(4, 2)
    bad = [
        lambda: kda.kda_layer_norm(x),  # not on a GPU
        lambda: kda.kda_layer_norm(x[0]), lambda: kda.kda_layer_norm(x.half()), lambda: kda.kda_layer_norm(x.t()),
        lambda: kda.kda_layer_norm(x, w[:7]), lambda: kda.kda_layer_norm(x, w.bfloat16()),
        lambda: kda.kda_layer_norm(x, w, w, y=torch.zeros(4, 9)),
        lambda: kda.kda_layer_norm_backward(x, x[:3], st), lambda: kda.kda_layer_norm_backward(x, x, st[:3]),
        lambda: kda.kda_layer_norm_backward(x, codes, st), lambda: kda.kda_layer_norm_backward(x, codes, st, x_scales=codes),
        lambda: kda.kda_layer_norm_backward(x, x, st, x_scales=scales),
        lambda: kda.kda_norm_layer(x, saved="fp8"),
        lambda: kda.kda_pack8(x[0]), lambda: kda.kda_pack8(x.double()), lambda: kda.kda_pack8(x),
        lambda: kda.kda_unpack8(codes, scales[:3]), lambda: kda.kda_unpack8(x, scales), lambda: kda.kda_unpack8(codes, scales),
        lambda: kda.kda_ssm_conv(x, torch.zeros(8, 3), [0, 4]), lambda: kda.kda_ssm_conv(x, torch.zeros(8, 4), [0, 4]),
        lambda: kda.kda_ssm_conv(x, torch.zeros(8, 4), [0, 4], conv_state_in=torch.zeros(1, 8, 2)),
        lambda: kda.kda_ssm_conv_step(x, torch.zeros(8, 4), None),
        lambda: kda.kda_ssm_conv_step(x, torch.zeros(8, 4), torch.zeros(3, 8, 3)),
        lambda: kda.kda_ssm_conv_step(x, torch.zeros(8, 4), torch.zeros(4, 8, 3)),
    ]
    A, B = torch.zeros(8, 16), torch.zeros(4, 1, 16)
    bad += [
        lambda: kda.kda_ssm_scan(x, x, A, B, B, [0, 4]), lambda: kda.kda_ssm_scan(x, x[:, :7], A, B, B, [0, 4]),
        lambda: kda.kda_ssm_scan(x, x, A[:7], B, B, [0, 4]), lambda: kda.kda_ssm_scan(x, x, A, B, B[:, :, :8], [0, 4]),
        lambda: kda.kda_ssm_scan(x, x, A, B.bfloat16(), B, [0, 4]),
        lambda: kda.kda_ssm_scan(x, x, A, B, B, [0, 4], initial_state=torch.zeros(2, 8, 16)),
        lambda: kda.kda_ssm_scan(x, x, A, B, B, [0, 4], D=torch.zeros(9)),
        lambda: kda.kda_ssm_step(x, x, A, B, B, None), lambda: kda.kda_ssm_step(x, x, A, B, B, torch.zeros(4, 8, 16)),
        lambda: kda.kda_ssm_step(x, x, A, B, B, torch.zeros(3, 8, 16)),
        lambda: kda.kda_ssm_backward(x, x, A, B, B, [0, 4], x[:3]),
        lambda: kda.kda_ssm_backward(x, x, A, B, B, [0, 4], x, d_final_state=torch.zeros(1, 8, 8)),
        lambda: kda.kda_ssm_layer(x, x, A, B, B, [0, 4], saved=""),
        lambda: kda.kda_ssm_conv_layer(x, torch.zeros(8, 4), [0, 4], saved=None),
        lambda: kda.kda_layer(None, None, None, None, None, None, None, saved="int8"),
    ]
    for i, f in enumerate(bad):
        with pytest.raises(ValueError):
            f()
            raise AssertionError(f"call {i} was accepted")


def test_packed_structs_are_the_declared_ones():
    """The packed formats lay every member of the C structs where their mirrors have it."""
    from kimi_delta_attention_16_gb300 import block

    def flat(cls, prefix=""):
        for name, typ in cls._fields_:
            if issubclass(typ, ctypes.Structure):
                yield from flat(typ, prefix + name + ".")
            else:
                yield prefix + name, typ

    for fmt, cls in ((block._NORM, _lib.NormArgs), (block._NORM_BWD, _lib.NormBackwardArgs), (block._CONV, _lib.SsmConvArgs),
                     (block._CONV_BWD, _lib.SsmConvBackwardArgs), (block._SSM, _lib.SsmArgs),
                     (block._SSM_BWD, _lib.SsmBackwardArgs)):
        names = list(flat(cls))
        values = [0.5 if t is ctypes.c_float else 1000 + i for i, (_, t) in enumerate(names)]
        got = cls.from_buffer_copy(fmt.pack(*values))
        assert fmt.size == ctypes.sizeof(cls)
        for (name, _), v in zip(names, values):
            obj = got
            for part in name.split("."):
                obj = getattr(obj, part)
            assert obj == v, name


def test_broadcast_rows_are_refused():
    """A stride of 0 means "dense" to the library, so a broadcast row would be read past its end."""
    row, rows = torch.zeros(1, 64).expand(8, 64), torch.zeros(8, 64)
    w, cu, A = torch.zeros(64, 4), torch.tensor([0, 8], dtype=torch.int32), torch.zeros(64, 16)
    BC, one = torch.zeros(8, 1, 16), torch.zeros(1, 1, 16).expand(8, 1, 16)
    stats = torch.zeros(8, 2)
    for call in (lambda: kda.kda_layer_norm(row), lambda: kda.kda_layer_norm(rows, y=row),
                 lambda: kda.kda_layer_norm_backward(row, rows, stats), lambda: kda.kda_layer_norm_backward(rows, row, stats),
                 lambda: kda.kda_pack8(row), lambda: kda.kda_pack8(torch.zeros(1, 1).expand(4, 1)),
                 lambda: kda.kda_ssm_conv(row, w, cu), lambda: kda.kda_ssm_conv_step(row, w, torch.zeros(8, 64, 3)),
                 lambda: kda.kda_ssm_conv_backward(rows, w, cu, row), lambda: kda.kda_ssm_scan(row, rows, A, BC, BC, cu),
                 lambda: kda.kda_ssm_scan(rows, rows, A, one, BC, cu), lambda: kda.kda_ssm_scan(rows, rows, A, BC, one, cu),
                 lambda: kda.kda_ssm_scan(rows, rows, A, BC, BC, cu, z=row),
                 lambda: kda.kda_ssm_step(rows, row, A, BC, BC, torch.zeros(8, 64, 16)),
                 lambda: kda.kda_ssm_backward(rows, rows, A, BC, BC, cu, row),
                 lambda: kda.kda_layer_norm(torch.zeros(4, 40).as_strided((8, 16), (8, 1)))):
        with pytest.raises(ValueError, match="overlap"):
            call()


def test_status_words_and_workspaces_are_checked():
    from kimi_delta_attention_16_gb300 import block
    assert block._status(None) == 0
    for bad in (torch.zeros(1, dtype=torch.int8), torch.zeros(0, dtype=torch.int32), torch.zeros(1)):
        with pytest.raises(ValueError, match="int32"):
            block._status(bad)
    wide = torch.zeros(1, dtype=torch.uint8).expand(1 << 20)  # claims a million bytes and has one
    with pytest.raises(ValueError, match="contiguous"):
        block._workspace("", 0, (), None, (), (), wide, None)


def test_scan_gradients_refuse_more_groups_than_a_grid_has_rows():
    n = ctypes.c_size_t(0)
    for groups, code in ((65536, UNSUPPORTED), (65535, 0)):
        a = ssm_bwd(fwd__G=groups, fwd__C=groups, fwd__T_total=0)
        assert _lib.load().kda_ssm_backward_workspace_size(ctypes.byref(a), ctypes.byref(n)) == code
    a = ssm_bwd(fwd__G=65536, fwd__C=65536)
    assert call("kda_ssm_backward", a) == UNSUPPORTED
