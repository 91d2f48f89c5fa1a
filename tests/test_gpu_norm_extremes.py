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
