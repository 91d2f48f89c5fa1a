"""How many digits the scan keeps in fp32: its step size, and its gradients where states forget quickly."""
import pytest
import torch

import kimi_delta_attention_16_gb300 as kda
from block_testlib import U32, gen, randn, ssm_inputs, within
from test_gpu_ssm import ref_grads, run_backward

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


def grad_errors(a, lens, dy, dfin):
    """Absolute error bounds of every gradient, carried along with the scan on magnitudes: each quantity's error is what its
    factors bring plus the roundings of its own operations, in units of 2^-24.

    step size (15 + 2 |x|: the test above, and the rounding of dt + dt_bias, which softplus hands on at most in full);
    decay: hardware exponential 4, log2 e and the product 3 |delta A|, the step size's error times |delta A|;
    gate and its slope: sigmoid (exponent |z|, exponential 4, sum and reciprocal 3) and up to five products (12 + 2 |z|);
    sums over states N, over channels Ch, over tokens: a piece's tokens one by one, then the pieces."""
    m = {k: (None if t is None else t.double().abs()) for k, t in a.items()}
    x = a["dt"].double() + a["dt_bias"].double()
    delta, slope = torch.logaddexp(x, torch.zeros_like(x)), torch.sigmoid(x)
    T, Ch = delta.shape
    G, N = a["B"].shape[1:]
    A, u, z = a["A"].double(), m["u"], a["z"].double()
    wide = lambda r: r.unsqueeze(1).expand(G, Ch // G, N).reshape(Ch, N)  # noqa: E731
    over = lambda v: v.view(G, Ch // G, N).sum(1)  # noqa: E731
    sg = torch.sigmoid(z)
    g, dsz = dy.double().abs() * (z * sg).abs(), sg * (1 + z.abs())
    rd, rg = (15 + 2 * x.abs()) * U32, (12 + 2 * z.abs()) * U32
    tokens = (72 + T // 64 + 16) * U32  # pieces of at most 72 tokens here
    out = {k: torch.zeros_like(v) for k, v in (("du", u), ("ddt", u), ("dz", u), ("dB", m["B"]), ("dC", m["C"]), ("dA", A))}
    dA = torch.zeros_like(A)
    out["dinitial_state"] = torch.zeros(len(lens), Ch, N, dtype=torch.float64)
    sums = {"dD": torch.zeros(Ch, dtype=torch.float64), "ddt_bias": torch.zeros(Ch, dtype=torch.float64)}
    out |= {k: torch.zeros_like(v) for k, v in sums.items()}
    t0 = 0
    for i, L in enumerate(lens):
        h, eh, hist = m["init"][i], torch.zeros(Ch, N, dtype=torch.float64), []
        for t in range(t0, t0 + L):
            hist.append((h, eh))
            E = (delta[t].unsqueeze(1) * A).abs()
            dec, rdec = torch.exp(-E), 5 * U32 + E * (3 * U32 + rd[t].unsqueeze(1))
            inp = (delta[t] * u[t]).unsqueeze(1) * wide(m["B"][t])
            eh = dec * (eh + h * rdec) + inp * (rd[t].unsqueeze(1) + 2 * U32)
            h = dec * h + inp
            eh = eh + U32 * h
        hist.append((h, eh))
        q, eq = dfin[i].double().abs(), torch.zeros(Ch, N, dtype=torch.float64)
        for t in range(t0 + L - 1, t0 - 1, -1):
            (h, eh), (hb, ehb) = hist[t - t0 + 1], hist[t - t0]
            d, r, gt, rt = (v[t].unsqueeze(1) for v in (delta, rd, g, rg))
            B, C, gu, du = wide(m["B"][t]), wide(m["C"][t]), g[t] * u[t], d * u[t].unsqueeze(1)
            E = d * A.abs()
            dec, rdec = torch.exp(-E), 5 * U32 + E * (3 * U32 + r)
            lam, el = q + gt * C, eq + gt * C * (rt + U32)
            el = el + U32 * lam
            out["dC"][t] = over(gt * (eh + h * (rt + (Ch + 1) * U32)))
            out["dB"][t] = over(du * (el + lam * (r + (Ch + 2) * U32)))
            q, eq = dec * lam, dec * (el + lam * (rdec + U32))
            w, ew = q * hb, eq * hb + q * ehb + U32 * q * hb
            dA += w * d
            out["dA"] += d * (ew + w * (r + 2 * U32))
            s1, e1 = (lam * B).sum(1), (B * (el + lam * (N + 1) * U32)).sum(1)
            s2, e2 = (w * A.abs()).sum(1), (A.abs() * (ew + w * (N + 4) * U32)).sum(1)
            D = m["D"]
            out["du"][t] = delta[t] * (e1 + s1 * (rd[t] + 2 * U32)) + D * g[t] * (rg[t] + 2 * U32)
            dd = u[t] * s1 + s2
            edd = (u[t] * e1 + e2 + 3 * U32 * dd) * slope[t] + dd * slope[t] * (10 + 2 * x[t].abs()) * U32
            out["ddt"][t] = edd
            yy = (C * h).sum(1)
            ey = (C * (eh + h * (N + 2) * U32)).sum(1)
            out["dz"][t] = dy[t].double().abs() * dsz[t] * (ey + (yy + D * u[t]) * (16 + 2 * z[t].abs()) * U32)
            sums["dD"] += gu
            out["dD"] += gu * (rg[t] + 2 * U32)
            sums["ddt_bias"] += dd * slope[t]
            out["ddt_bias"] += edd
        out["dinitial_state"][i] = eq
        t0 += L
    out["dA"] += tokens * dA
    for k, v in sums.items():
        out[k] += tokens * v
    return out


@pytest.mark.parametrize("lens", [[1500], [640, 0, 260, 600]])
@pytest.mark.parametrize("N,G", [(8, 1), (16, 1), (32, 2), (64, 1)])
def test_gradients_of_states_that_forget(lens, N, G):
    """Step sizes of 0.1 to 0.5, so that a state lasts a few tokens and the bounds stay at tens of units however long the
    sequence is."""
    T, n, Ch = sum(lens), len(lens), 16
    a = ssm_inputs(T + N, T, Ch, N, G, torch.float32, n)
    g = gen(T)
    step = 0.1 + 0.4 * torch.rand(Ch, generator=g)
    a["dt_bias"] = step + torch.log(-torch.expm1(-step))
    dy, dfin = randn(g, T, Ch), randn(g, n, Ch, N)
    got, ref, tol = run_backward(a, lens, dy, dfin), ref_grads(a, lens, dy, dfin), grad_errors(a, lens, dy, dfin)
    assert set(got) == set(ref) == set(tol)
    for name, r in ref.items():
        within(got[name], r, tol[name] + U32 * r.abs(), name)
