"""The scan and its gradients where sequences end exactly where the pieces of the token axis do (64 tokens each here)."""
import pytest
import torch

from block_testlib import U32, gen, randn, ssm_inputs, ssm_ref, within
from test_gpu_ssm import grad_bounds, ref_grads, run_backward, run_scan, scan_bounds

pytestmark = pytest.mark.gpu
FP = torch.float32
PER_TOKEN = ("du", "ddt", "dz", "dB", "dC")  # of one sequence alone, like dinitial_state


@pytest.mark.parametrize("lens", [[512] * 4, [300, 724, 1024], [1024, 0, 1024], [64, 192, 0, 0, 1792]])
@pytest.mark.parametrize("N,G,dfinal", [(8, 1, True), (16, 1, True), (16, 2, False), (32, 1, True), (64, 1, False)])
def test_border_of_a_sequence_on_the_border_of_a_piece(lens, N, G, dfinal):
    """Slow decays, so that whatever crossed a border would be seen a thousand tokens away."""
    T, n, Ch = sum(lens), len(lens), 8
    a = ssm_inputs(T + N, T, Ch, N, G, FP, n, slow=True)
    y, fin = run_scan(a, lens)
    ry, rf = ssm_ref(a["u"], a["dt"], a["A"], a["B"], a["C"], lens, a["D"], a["z"], a["dt_bias"], True, a["init"])
    ey, ef = scan_bounds(a, lens)
    within(y, ry, ey + U32 * ry.abs(), "y")
    within(fin, rf, ef, "final_state")
    g = gen(T + 1)
    dy, dfin = randn(g, T, Ch), (randn(g, n, Ch, N) if dfinal else None)
    got = run_backward(a, lens, dy, dfin)
    ref, tol = ref_grads(a, lens, dy, dfin), grad_bounds(a, lens, dy, dfin)
    for name, r in ref.items():
        within(got[name], r, tol[name] + U32 * r.abs(), name)


@pytest.mark.parametrize("lens", [[512] * 4, [300, 724, 1024], [1024, 0, 1024], [64, 192, 0, 0, 1792], [700, 648, 700]])
@pytest.mark.parametrize("N", [8, 16, 32, 64])
def test_later_sequences_do_not_reach_earlier_ones(lens, N):
    """Other gradients at a later sequence's outputs and final state leave the earlier sequences' own gradients as they
    are, bit by bit; so does other input in an earlier sequence the later ones' outputs."""
    T, n, Ch = sum(lens), len(lens), 24
    a = ssm_inputs(T + N, T, Ch, N, 1, FP, n, slow=True)
    g = gen(T + 2)
    dy, dfin = randn(g, T, Ch), randn(g, n, Ch, N)
    got, (y, fin) = run_backward(a, lens, dy, dfin), run_scan(a, lens)
    for first in range(1, n):
        at = sum(lens[:first])
        dy2, dfin2 = dy.clone(), dfin.clone()
        dy2[at:], dfin2[first:] = 1e6, float("nan")
        other = run_backward(a, lens, dy2, dfin2)
        for name in PER_TOKEN:
            assert torch.equal(other[name][:at], got[name][:at]), (name, first)
        assert torch.equal(other["dinitial_state"][:first], got["dinitial_state"][:first]), first
        b = dict(a, u=a["u"].clone(), init=a["init"].clone())
        b["u"][:at], b["init"][:first] = 1e6, float("nan")
        y2, fin2 = run_scan(b, lens)
        assert torch.equal(y2[at:], y[at:]) and torch.equal(fin2[first:], fin[first:]), first
