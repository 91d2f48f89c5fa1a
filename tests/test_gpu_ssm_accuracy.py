"""How many digits the scan keeps in fp32."""
import pytest
import torch

import kimi_delta_attention_16_gb300 as kda
from block_testlib import U32, gen, within

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.mark.parametrize("step", [False, True])
def test_step_size_is_softplus_to_a_dozen_units(step):
    """One token from a zero state with u = 1 and B = (1, 0, ..) leaves the step size itself as the state.  In units of
    2^-24, relative: the hardware exponential 4, its correction 1, log 2's own rounding |x| / 21, the sum 2 + e 1, the
    hardware reciprocal 2, a product 1, the polynomial 1.6, the last multiply-add 1."""
    Ch = 1 << 16
    x = torch.rand(1, Ch, generator=gen(1)) * 105 - 85
    x[0, :6] = torch.tensor([0.0, -0.0, 3e38, -3e38, float("inf"), float("-inf")])
    one, A = torch.ones(1, Ch), -torch.ones(Ch, 8)
    B = torch.zeros(1, 1, 8)
    B[0, 0, 0] = 1.0
    args = [t.to(DEV) for t in (one, x, A, B, B)]
    if step:
        state = torch.zeros(1, Ch, 8, device=DEV)
        kda.kda_ssm_step(*args, state)
    else:
        _, state = kda.kda_ssm_scan(*args, [0, 1])
    got, xs = state[0, 6:, 0], x[0, 6:].double()
    ref = torch.logaddexp(xs, torch.zeros_like(xs))
    within(got, ref, (12 + xs.abs() / 20) * U32 * ref, "step size")
    ends = state[0, :6, 0].cpu()
    assert (ends[:2] - 0.6931472).abs().max() < 1e-6 and ends[2] == x[0, 2] and ends[4] == x[0, 4]
    assert ends[3] == 0 and ends[5] == 0
    x[0, 9] = float("nan")
    y, state = kda.kda_ssm_scan(args[0], x.to(DEV), *args[2:], [0, 1])
    assert torch.isnan(state[0, 9, 0]) and torch.isfinite(state[0, 6:9]).all() and torch.isfinite(state[0, 10:]).all()
