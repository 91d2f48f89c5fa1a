"""Layer norm and 8-bit activations on the GPU against plain 64-bit forms."""
import pytest
import torch

import kimi_delta_attention_16_gb300 as kda
from block_testlib import U, U32, f64, gen, norm_ref, pack8_ref, randn, within

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF, FP = torch.bfloat16, torch.float32


def rows_in(t, how):
    """t on the GPU as a dense tensor, as rows of a wider buffer, or one element off alignment."""
    t = t.to(DEV)
    if how == "dense":
        return t
    pad, off = (8, 0) if how == "strided" else (3, 1)
    buf = torch.full((t.shape[0], t.shape[1] + pad), float("nan"), dtype=t.dtype, device=DEV)
    view = buf[:, off:off + t.shape[1]]
    view.copy_(t)
    return view


def norm_bounds(x, ref, w, b, dy=None, xb=None):
    """fp32 error bounds of one row pass.  A sum over C values by threads and shuffles rounds at most 44 times along any
    path (32 elements a thread, ten shuffle levels, two more), each time by 2^-24 of a partial sum of magnitudes."""
    c = 44 * U32
    x, r = f64(x), ref["rstd"].unsqueeze(1)
    w = torch.ones(x.shape[1], dtype=torch.float64) if w is None else f64(w).abs()
    b = torch.zeros(x.shape[1], dtype=torch.float64) if b is None else f64(b).abs()
    dmean = c * x.abs().mean(1, keepdim=True)  # of the mean
    # of xh: the mean's, one subtraction, rstd's relative error (var twice that of a deviation, plus its sum) on |xh|
    xh = ((x - ref["mean"].unsqueeze(1)) * r).abs()
    drel = c + 2 * (dmean * r) * 2 + 8 * U32
    dxh = (dmean + 2 * U32 * x.abs()) * r + xh * drel
    out = {"y": dxh * w + 3 * U32 * (xh * w + b)}
    if dy is not None:
        dy = f64(dy)
        hb = ((f64(xb if xb is not None else x) - ref["mean"].unsqueeze(1)) * r).abs()
        dhb = (dmean + 2 * U32 * f64(xb if xb is not None else x).abs()) * r + hb * drel
        p = (dy * w).abs()
        m0, m1 = p.mean(1, keepdim=True), (p * hb).mean(1, keepdim=True)
        dm1 = (p * dhb).mean(1, keepdim=True) + c * m1
        out["dx"] = r * (4 * U32 * p + c * m0 + dhb * m1 + hb * dm1 + 4 * U32 * hb * m1) + r * drel * (p + m0 + hb * m1)
        k = (x.shape[0] + 64) * U32  # column sums: at most one rounding per row, and the joins
        out["dweight"] = (dy.abs() * dhb).sum(0) + k * (dy.abs() * hb).sum(0)
        out["dbias"] = k * dy.abs().sum(0)
    return out


@pytest.mark.parametrize("io", [BF, FP])
@pytest.mark.parametrize("M,C,how", [
    (1, 1, "dense"), (3, 7, "dense"), (5, 64, "dense"), (2, 1000, "dense"), (300, 1001, "dense"), (4, 1024, "strided"),
    (7, 4096, "dense"), (3, 7168, "odd"), (2, 16384, "dense"), (2, 16392, "dense"), (1, 32768, "dense"),
    (2, 32767, "dense"), (1300, 96, "dense"), (700, 8, "strided")])
@pytest.mark.parametrize("saved", ["io", "e4m3"])
def test_layer_norm_and_gradient(M, C, how, io, saved):
    g = gen(M * 1000 + C)
    x = (randn(g, M, C) * 3 + randn(g, M, 1) * 5).to(io)  # rows with means of their own
    w, b, dy = randn(g, C, std=0.3, mean=1.0), randn(g, C, std=0.3), randn(g, M, C, dtype=io)
    xg, dyg = rows_in(x, how), rows_in(dy, how)
    y, stats = kda.kda_layer_norm(xg, w.to(DEV), b.to(DEV), eps=1e-5, return_stats=True)
    xs, scales, xb = (xg, None, None)
    if saved == "e4m3":
        (xs, scales), xb = kda.kda_pack8(xg), pack8_ref(x)[0]
    got = kda.kda_layer_norm_backward(dyg, xs, stats, w.to(DEV), x_scales=scales)
    ref = norm_ref(x, w, b, 1e-5, dy, xb)
    tol = norm_bounds(x, ref, w, b, dy, xb)
    u = U[io]
    within(y, ref["y"], tol["y"] + u * (ref["y"].abs() + tol["y"]), "y")
    within(got["dx"], ref["dx"], tol["dx"] + u * (ref["dx"].abs() + tol["dx"]), "dx")
    within(got["dweight"], ref["dweight"], tol["dweight"], "dweight")
    within(got["dbias"], ref["dbias"], tol["dbias"], "dbias")
    again = kda.kda_layer_norm_backward(dyg, xs, stats, w.to(DEV), x_scales=scales)
    assert all(torch.equal(got[k], again[k]) for k in got)  # fixed order of the sums


@pytest.mark.parametrize("io", [BF, FP])
@pytest.mark.parametrize("M,C", [(5000, 96), (4900, 520), (2600, 1800), (1500, 2048), (1300, 4096), (1300, 7168), (700, 8192),
                                 (650, 14336)])
def test_layer_norm_many_rows(M, C, io):
    """Enough rows for every SM to take several in turn, at each width class, without a weight in the odd ones."""
    g = gen(M + C)
    x, dy = (randn(g, M, C) * 3 + randn(g, M, 1) * 5).to(io), randn(g, M, C, dtype=io)
    w, b = (randn(g, C, std=0.3, mean=1.0), randn(g, C, std=0.3)) if C % 1000 else (None, None)
    put = lambda t: None if t is None else t.to(DEV)  # noqa: E731
    y, stats = kda.kda_layer_norm(x.to(DEV), put(w), put(b), return_stats=True)
    got = kda.kda_layer_norm_backward(dy.to(DEV), x.to(DEV), stats, put(w))
    ref = norm_ref(x, w, b, 1e-5, dy)
    tol, u = norm_bounds(x, ref, w, b, dy), U[io]
    within(y, ref["y"], tol["y"] + u * (ref["y"].abs() + tol["y"]), "y")
    within(got["dx"], ref["dx"], tol["dx"] + u * (ref["dx"].abs() + tol["dx"]), "dx")
    within(got["dweight"], ref["dweight"], tol["dweight"], "dweight")
    within(got["dbias"], ref["dbias"], tol["dbias"], "dbias")
    again = kda.kda_layer_norm(x.to(DEV), put(w), put(b))
    few = kda.kda_layer_norm(x[:5].to(DEV), put(w), put(b))
    assert torch.equal(again, y)
    within(few, ref["y"][:5], (tol["y"] + u * (ref["y"].abs() + tol["y"]))[:5], "five rows")


def test_layer_norm_without_parameters_and_large_mean():
    g = gen(3)
    x = randn(g, 9, 512) + 1000.0  # a two-pass variance keeps its digits: one pass of squares would lose six
    y, stats = kda.kda_layer_norm(x.to(DEV), return_stats=True)
    ref = norm_ref(x, None, None, 1e-5)
    tol = norm_bounds(x, ref, None, None)["y"]
    within(y, ref["y"], tol + U32 * ref["y"].abs(), "y")
    dy = randn(g, 9, 512)
    got = kda.kda_layer_norm_backward(dy.to(DEV), x.to(DEV), stats, param_grads=False)
    assert set(got) == {"dx"}


def test_layer_norm_rows_stand_alone():
    """A NaN or infinity in one row stays there; constant rows give the bias; no rows give zero parameter gradients."""
    g = gen(4)
    x, w, b = randn(g, 5, 200), randn(g, 200), randn(g, 200)
    clean = kda.kda_layer_norm(x.to(DEV), w.to(DEV), b.to(DEV))
    x[1, 3], x[2, 7] = float("nan"), float("inf")
    x[4] = 2.5
    y = kda.kda_layer_norm(x.to(DEV), w.to(DEV), b.to(DEV))
    assert torch.equal(y[0], clean[0]) and torch.equal(y[3], clean[3])
    assert torch.isnan(y[1]).all() and torch.isnan(y[2]).all()
    assert torch.equal(y[4].cpu(), b)
    none = torch.empty(0, 200, device=DEV)
    y, stats = kda.kda_layer_norm(none, w.to(DEV), b.to(DEV), return_stats=True)
    got = kda.kda_layer_norm_backward(none, none, stats, w.to(DEV))
    assert y.shape == (0, 200) and not got["dweight"].any() and not got["dbias"].any()


@pytest.mark.parametrize("saved", ["io", "e4m3"])
def test_norm_layer_gradients_and_graph(saved):
    """The autograd form gives the direct calls' gradients, and its step can be captured and replayed."""
    g = gen(5)
    x = randn(g, 64, 320, dtype=BF).to(DEV).requires_grad_()
    w = randn(g, 320).to(DEV).requires_grad_()
    b = randn(g, 320).to(DEV).requires_grad_()
    dy = randn(g, 64, 320, dtype=BF).to(DEV)
    y = kda.kda_norm_layer(x, w, b, saved=saved)
    dx, dw, db = torch.autograd.grad(y, (x, w, b), dy)
    _, stats = kda.kda_layer_norm(x.detach(), w.detach(), b.detach(), return_stats=True)
    xs, sc = kda.kda_pack8(x.detach()) if saved == "e4m3" else (x.detach(), None)
    ref = kda.kda_layer_norm_backward(dy, xs, stats, w.detach(), x_scales=sc)
    assert torch.equal(dx, ref["dx"]) and torch.equal(dw, ref["dweight"]) and torch.equal(db, ref["dbias"])
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=side):
        yc, st = kda.kda_layer_norm(x.detach(), w.detach(), b.detach(), return_stats=True)
        xs, sc = kda.kda_pack8(x.detach()) if saved == "e4m3" else (x.detach(), None)
        cap = kda.kda_layer_norm_backward(dy, xs, st, w.detach(), x_scales=sc)
    with torch.no_grad():
        x.mul_(-2.0)
    graph.replay()
    torch.cuda.synchronize()
    y2, st2 = kda.kda_layer_norm(x.detach(), w.detach(), b.detach(), return_stats=True)
    assert torch.equal(yc, y2) and torch.equal(st, st2)
    xs, sc = kda.kda_pack8(x.detach()) if saved == "e4m3" else (x.detach(), None)
    ref = kda.kda_layer_norm_backward(dy, xs, st2, w.detach(), x_scales=sc)
    assert all(torch.equal(cap[k], ref[k]) for k in ref)


@pytest.mark.parametrize("io", [BF, FP])
@pytest.mark.parametrize("M,C,how", [(1, 1, "dense"), (3, 31, "dense"), (5, 33, "dense"), (9, 64, "strided"),
                                     (4, 1000, "odd"), (6, 2056, "dense"), (1000, 96, "dense"), (2, 12288, "dense")])
def test_pack8_is_the_definition(M, C, how, io):
    """Codes and scales equal the definition bit by bit, and so do the values read back (every one of them exact)."""
    g = gen(M + C)
    x = (randn(g, M, C) * torch.exp2(torch.randint(-20, 20, (M, C), generator=g).float())).to(io)
    x[0, 0] = 448.0  # a block whose largest value is exactly the largest code
    if C >= 64:
        x[-1, 32:64] = 0.0
    if C > 600:
        x[0, 64:96] = 1e-37 * randn(g, 32)
    xg = rows_in(x, how)
    codes, scales = kda.kda_pack8(xg)
    values, bytes_ = pack8_ref(x)
    assert torch.equal(scales.cpu(), bytes_)
    back = kda.kda_unpack8(codes, scales, dtype=FP)
    assert torch.equal(back.cpu().double(), values)
    # half a step of e4m3, or half the smallest step under the block's scale
    s = torch.exp2(bytes_.double() - 127).repeat_interleave(32, 1)[:, :C]
    within(back, x, torch.maximum(2.0 ** -4 * f64(x).abs(), 2.0 ** -10 * s), "half a step")
    out = rows_in(torch.zeros(M, C, dtype=io), how)
    kda.kda_unpack8(codes, scales, out=out)
    assert torch.equal(out.cpu().double(), values.to(io).double())


def test_pack8_keeps_what_is_not_finite():
    x = torch.ones(3, 96)
    x[0, 5], x[0, 40], x[1, 70] = float("nan"), float("inf"), float("-inf")
    x[2, :32] = float("nan")  # a block with nothing finite in it
    back = kda.kda_unpack8(*kda.kda_pack8(x.to(DEV)), dtype=FP)
    within(back, pack8_ref(x)[0], 0.0)
    assert torch.isnan(back.cpu()[0, 40]) and torch.isnan(back.cpu()[1, 70])
    empty = kda.kda_pack8(torch.empty(0, 40, device=DEV))
    assert empty[0].shape == (0, 40) and empty[1].shape == (0, 2)


def test_pack8_on_another_stream():
    x = randn(gen(8), 512, 2048, dtype=BF).to(DEV)
    ref = kda.kda_pack8(x)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    codes, scales = kda.kda_pack8(x, stream=s)
    back = kda.kda_unpack8(codes, scales, stream=s.cuda_stream)
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda.synchronize()
    assert torch.equal(codes, ref[0]) and torch.equal(scales, ref[1])
    assert torch.equal(back, kda.kda_unpack8(*ref))
