"""Layer norm of rows at the ends of fp32's range and of rows whose mean is far above their deviation."""
import pytest
import torch

import kimi_delta_attention_16_gb300 as kda
from block_testlib import U32, gen, randn, within

pytestmark = pytest.mark.gpu
DEV, BF, FP = "cuda", torch.bfloat16, torch.float32


@pytest.mark.parametrize("C", [96, 333, 4096])  # rows through shared memory, single elements, four accesses per thread
@pytest.mark.parametrize("eps", [1e-5, 0.0])
def test_a_row_does_not_depend_on_the_rows_beside_it(C, eps):
    """Rows whose variance overflows fp32, is zero or lies below its normal numbers, among five rows and among five
    thousand: the same kind of result, and the bias where the deviation's reciprocal is 0."""
    g = gen(C)
    x, w, b = randn(g, 5000, C), randn(g, C), randn(g, C)
    sign = 1.0 - 2.0 * (torch.arange(C) % 2)
    x[1], x[2], x[3] = 3e20 * sign, 2.5, 1e-21 * sign
    put = [t.to(DEV) for t in (w, b)]
    many, sm = kda.kda_layer_norm(x.to(DEV), *put, eps=eps, return_stats=True)
    few, sf = kda.kda_layer_norm(x[:5].to(DEV), *put, eps=eps, return_stats=True)
    assert torch.equal(sm[1, 1].cpu(), torch.tensor(0.0)) and torch.equal(sf[1, 1].cpu(), torch.tensor(0.0))
    assert torch.equal(many[1].cpu(), b) and torch.equal(few[1].cpu(), b)
    assert torch.equal(sm[2, 1].isinf(), sf[2, 1].isinf()) and sm[2, 1].isinf().item() == (eps == 0.0)
    # the two ways of summing C squares and of taking the root differ by at most (C + 8) roundings each
    for i in (0, 3, 4):
        within(sm[i, 1], sf[i, 1], 2 * (C + 8) * U32 * f_abs(sf[i, 1]), f"row {i}")
    dy = randn(g, 5000, C)
    dm = kda.kda_layer_norm_backward(dy.to(DEV), x.to(DEV), sm, put[0])["dx"]
    df = kda.kda_layer_norm_backward(dy[:5].to(DEV), x[:5].to(DEV), sf, put[0])["dx"]
    assert not dm[1].any() and not df[1].any()  # the row's output does not move
    assert torch.equal(dm[:5].isnan(), df.isnan())


def f_abs(t):
    return t.detach().cpu().double().abs()


@pytest.mark.parametrize("deviations", [100, 1000, 10000])
@pytest.mark.parametrize("saved", ["io", "e4m3"])
@pytest.mark.parametrize("M,C", [(9, 512), (5000, 512), (1300, 4096), (9, 333), (5000, 333), (40, 14340)])
def test_gradient_of_rows_with_a_large_mean(M, C, saved, deviations):
    """The backward pass on its own inputs: xh = (x - mean) rstd from the statistics it is given, in 64 bits.  In fp32 the
    subtraction and the product round xh twice, whatever the mean: 2 units of 2^-24 of |x - mean| rstd (8-bit x: its
    value is exact).  p = dy w rounds once; a sum of C terms over threads, shuffles and warps at most 44 times on any path;
    dx adds four more roundings of each of its three terms; a column sum one per row and 64 for the joins.  x rstd - mean rstd
    in one step would be off by the mean's deviations times 2^-24 instead."""
    g = gen(M + C + deviations)
    x = (randn(g, M, C) + deviations * (1 + randn(g, M, 1).abs())).to(FP)
    w, dy = randn(g, C, std=0.3, mean=1.0), randn(g, M, C)
    xg = x.to(DEV)
    _, stats = kda.kda_layer_norm(xg, w.to(DEV), return_stats=True)
    xs, scales, xb = xg, None, x.double()
    if saved == "e4m3":
        xs, scales = kda.kda_pack8(xg)
        xb = kda.kda_unpack8(xs, scales, dtype=FP).cpu().double()  # exact
    got = kda.kda_layer_norm_backward(dy.to(DEV), xs, stats, w.to(DEV), x_scales=scales)
    mean, rstd = (t.unsqueeze(1) for t in stats.cpu().double().unbind(1))
    dy, w = dy.double(), w.double()
    xh, p = (xb - mean) * rstd, dy * w
    m0, m1 = p.mean(1, keepdim=True), (p * xh).mean(1, keepdim=True)
    a0, a1, h = p.abs().mean(1, keepdim=True), (p * xh).abs().mean(1, keepdim=True), xh.abs()
    e0, e1 = 46 * U32 * a0, 50 * U32 * a1
    within(got["dx"], rstd * (p - m0 - xh * m1), rstd * (5 * U32 * (p.abs() + a0 + h * a1) + e0 + h * e1), "dx")
    k = (M + 64 + 3) * U32
    within(got["dweight"], (dy * xh).sum(0), k * (dy * xh).abs().sum(0), "dweight")
    within(got["dbias"], dy.sum(0), k * dy.abs().sum(0), "dbias")
