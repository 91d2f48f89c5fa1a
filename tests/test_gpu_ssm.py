"""The selective state space scan and its short convolution on the GPU against plain 64-bit forms."""
import pytest
import torch

import kimi_delta_attention_16_gb300 as kda
from block_testlib import U, U32, conv_ref, f64, gen, randn, ssm_inputs, ssm_ref, within
from test_gpu_norm_pack8 import rows_in

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF, FP = torch.bfloat16, torch.float32


def cu_of(lens):
    cu = [0]
    for L in lens:
        cu.append(cu[-1] + L)
    return cu


def to(t):
    return None if t is None else t.to(DEV)


# ------------------------------------------------------------------ the short convolution
CONV_LENS = [[1], [2], [3], [4], [0, 5, 0, 0, 1, 2, 3, 40, 0], [7, 8, 9, 64, 63, 65], [300, 1, 129], [1] * 40]


def conv_bounds(x, w, bias, dy, lens, state):
    """Five roundings of the sum, then SiLU to at most 16 units of the last place (an exponential, a division and two
    products); its derivative amplifies the sum's error by at most 1.1, and its own slope by 0.5."""
    mag = conv_ref(x.abs(), w.abs(), None if bias is None else bias.abs(), lens, False,
                   None if state is None else state.abs())["y"]  # sum of the terms' magnitudes
    return {"y": 2 * 5 * U32 * mag + 16 * U32 * mag, "dpre": dy.double().abs() * (20 * U32 * (1 + mag))}


@pytest.mark.parametrize("lens", CONV_LENS)
@pytest.mark.parametrize("C,how,io", [(64, "dense", BF), (40, "strided", BF), (33, "dense", BF), (300, "odd", BF),
                                      (64, "dense", FP), (31, "dense", FP), (1028, "strided", FP)])
@pytest.mark.parametrize("state,silu", [(True, True), (False, True), (True, False)])
def test_conv_and_gradient(lens, C, how, io, state, silu):
    T, n = sum(lens), len(lens)
    g = gen(T * 7 + C)
    x, dy = randn(g, T, C, dtype=io), randn(g, T, C, dtype=io)
    w, bias = randn(g, C, 4, std=0.5), randn(g, C, std=0.2)
    st = randn(g, n, C, 3, dtype=io) if state else None
    cu = cu_of(lens)
    xg, dyg = rows_in(x, how), rows_in(dy, how)
    y, last = kda.kda_ssm_conv(xg, to(w), cu, bias=to(bias), silu=silu, conv_state_in=to(st), output_conv_state=True)
    got = kda.kda_ssm_conv_backward(xg, to(w), cu, dyg, bias=to(bias), silu=silu, conv_state_in=to(st))
    ref = conv_ref(x, w, bias, lens, silu, st, dy)
    tol = conv_bounds(x, w, bias, dy, lens, st)
    u = U[io]
    within(y, ref["y"], tol["y"] + u * (ref["y"].abs() + tol["y"]), "y")
    assert torch.equal(last.cpu().double(), ref["state"])
    # the gradients are sums of dpre (its error bounded above) with four taps, or over the tokens
    bd = conv_ref(x.abs(), w.abs(), None, lens, False, None if st is None else st.abs(), tol["dpre"] + 1e-30)
    mag = conv_ref(x.abs(), w.abs(), None, lens, False, None if st is None else st.abs(), 1.2 * dy.double().abs())
    k = (T + 80) * U32
    within(got["dx"], ref["dx"], bd["dx"] + 4 * U32 * mag["dx"] + u * (ref["dx"].abs() + bd["dx"]), "dx")
    within(got["dw"], ref["dw"], bd["dw"] + k * mag["dw"], "dw")
    within(got["dbias"], ref["dbias"], bd["dbias"] + k * mag["dbias"], "dbias")
    if state:
        within(got["dconv_state_in"], ref["dstate"], bd["dstate"] + 4 * U32 * mag["dstate"], "dconv_state_in")
    else:
        assert "dconv_state_in" not in got


def test_conv_long_stream_in_pieces():
    """Many runs per sequence, runs that end inside one, and a device-only cu_seqlens."""
    lens = [2500, 0, 1, 1700, 4096, 3]
    T, C = sum(lens), 256
    g = gen(5)
    x, dy, w = randn(g, T, C, dtype=BF), randn(g, T, C, dtype=BF), randn(g, C, 4, std=0.5)
    y = kda.kda_ssm_conv(to(x), to(w), cu_of(lens), check_cu_on_host=False)
    got = kda.kda_ssm_conv_backward(to(x), to(w), cu_of(lens), to(dy), check_cu_on_host=False)
    ref = conv_ref(x, w, None, lens, True, None, dy)
    mag = conv_ref(x.abs(), w.abs(), None, lens, False, None, dy.double().abs() * 1.2)
    within(y, ref["y"], 30 * U32 * mag["y"] + U[BF] * ref["y"].abs() * 1.001, "y")
    within(got["dx"], ref["dx"], 60 * U32 * mag["dx"] * 8 + U[BF] * ref["dx"].abs() * 1.001, "dx")
    within(got["dw"], ref["dw"], (T + 200) * U32 * mag["dw"], "dw")
    again = kda.kda_ssm_conv_backward(to(x), to(w), cu_of(lens), to(dy), check_cu_on_host=False)
    assert all(torch.equal(got[k], again[k]) for k in got)


@pytest.mark.parametrize("io", [BF, FP])
@pytest.mark.parametrize("n,C", [(1, 1), (3, 33), (5, 256), (70, 1000)])
def test_conv_steps_continue_a_prompt(n, C, io):
    """A prompt's conv state, then three single-token steps, equal one longer prompt bit by bit."""
    g = gen(n + C)
    lens = [4 + i % 5 for i in range(n)]
    x = randn(g, sum(lens) + 3 * n, C, dtype=io)
    w, bias = randn(g, C, 4), randn(g, C)
    whole = [L + 3 for L in lens]
    cu = cu_of(whole)
    full, last = kda.kda_ssm_conv(to(x), to(w), cu, bias=to(bias), output_conv_state=True)
    head = torch.cat([x[cu[i]:cu[i] + lens[i]] for i in range(n)])
    _, st = kda.kda_ssm_conv(to(head), to(w), cu_of(lens), bias=to(bias), output_conv_state=True)
    for k in range(3):
        rows = torch.tensor([cu[i] + lens[i] + k for i in range(n)])
        y = kda.kda_ssm_conv_step(to(x[rows]), to(w), st, bias=to(bias))
        assert torch.equal(y, full[rows.to(DEV)])
    assert torch.equal(st, last)


# ------------------------------------------------------------------ the scan
def scan_bounds(a, lens, softplus=True):
    """Error bounds of y and the final state, as the scan run on magnitudes: each step's terms come with a relative error
    of r (step size 8 units of the last place, product and sum), and the decay with 3 units plus the step size's error times
    the exponent; over a state's memory those add up, which running the recurrence on |h| with those errors bounds."""
    f = {k: f64(v) for k, v in a.items()}
    x = f["dt"] if a["dt_bias"] is None else f["dt"] + f["dt_bias"]
    delta = (torch.logaddexp(x, torch.zeros_like(x)) if softplus else x).abs()
    T, Ch = f["u"].shape
    N, G = a["A"].shape[1], a["B"].shape[1]
    wide = lambda r: r.abs().unsqueeze(1).expand(G, Ch // G, N).reshape(Ch, N)  # noqa: E731
    A = f["A"]
    ey, ef, t = torch.zeros(T, Ch, dtype=torch.float64), [], 0
    rd = (8 + 2 * (x.abs() + 1)) * U32  # of delta: its exponential's argument is rounded too
    for i, L in enumerate(lens):
        h = torch.zeros(Ch, N, dtype=torch.float64) if a["init"] is None else f["init"][i].abs()
        e = torch.zeros_like(h)
        for t in range(t, t + L):
            dA = delta[t].unsqueeze(1) * A
            dec = torch.exp(dA)
            inp = (delta[t] * f["u"][t].abs()).unsqueeze(1) * wide(f["B"][t])
            rdec = 4 * U32 + dA.abs() * (rd[t].unsqueeze(1) + 3 * U32)
            e = dec * (e + h * (rdec + U32)) + inp * (rd[t].unsqueeze(1) + 4 * U32)
            h = dec * h + inp
            yy = (wide(f["C"][t]) * h).sum(1)
            ey[t] = (wide(f["C"][t]) * e).sum(1) + (N + 4) * U32 * (yy + (0 if a["D"] is None else (f["D"] * f["u"][t]).abs()))
        t = t + 1 if L else t
        ef.append(e + U32 * h)
    if a["z"] is not None:
        sz = (f["z"] * torch.sigmoid(f["z"])).abs()
        y = ssm_ref(a["u"], a["dt"], a["A"], a["B"], a["C"], lens, a["D"], None, a["dt_bias"], softplus, a["init"])[0]
        ey = ey * sz + y.abs() * sz * (10 + 2 * f["z"].abs()) * U32
    return ey, torch.stack(ef)


def run_scan(a, lens, how="dense", **kw):
    v = {k: (rows_in(t, how) if k in ("u", "dt", "z") and t is not None else to(t)) for k, t in a.items()}
    return kda.kda_ssm_scan(v["u"], v["dt"], v["A"], v["B"], v["C"], cu_of(lens), D=v["D"], z=v["z"],
                            dt_bias=v["dt_bias"], initial_state=v["init"], **kw)


SCAN_LENS = [[1], [15, 17], [0, 16, 0, 32, 1, 0], [5, 0, 11, 48, 1, 1, 1, 33], [130], [400, 3, 700]]


@pytest.mark.parametrize("lens", SCAN_LENS)
@pytest.mark.parametrize("Ch,N,G,how,io", [
    (64, 16, 1, "dense", BF), (64, 16, 1, "dense", FP), (40, 8, 2, "odd", BF), (1, 16, 1, "dense", FP),
    (96, 32, 3, "strided", BF), (130, 64, 2, "dense", FP), (200, 16, 1, "odd", FP), (129, 64, 1, "dense", BF)])
def test_scan(lens, Ch, N, G, how, io):
    T = sum(lens)
    a = ssm_inputs(T + Ch + N, T, Ch, N, G, io, len(lens), gate=Ch != 40, skip=Ch != 96, state=Ch != 200)
    y, fin = run_scan(a, lens, how)
    ry, rf = ssm_ref(a["u"], a["dt"], a["A"], a["B"], a["C"], lens, a["D"], a["z"], a["dt_bias"], True, a["init"])
    ey, ef = scan_bounds(a, lens)
    within(y, ry, ey + U[io] * (ry.abs() + ey), "y")
    within(fin, rf, ef, "final_state")


@pytest.mark.parametrize("softplus,bias", [(False, True), (True, False), (False, False)])
def test_scan_step_size_forms(softplus, bias):
    a = ssm_inputs(11, 90, 48, 16, 1, FP, 2, bias=bias)
    if not softplus:
        a["dt"] = a["dt"].abs() * 0.1
        if bias:
            a["dt_bias"] = a["dt_bias"].abs() * 0.01
    lens = [50, 40]
    y, fin = run_scan(a, lens, softplus=softplus)
    ry, rf = ssm_ref(a["u"], a["dt"], a["A"], a["B"], a["C"], lens, a["D"], a["z"], a["dt_bias"], softplus, a["init"])
    ey, ef = scan_bounds(a, lens, softplus)
    within(y, ry, ey + U32 * ry.abs(), "y")
    within(fin, rf, ef, "final_state")


def test_scan_slow_decay_over_pieces():
    """States that remember a thousand tokens, through every piece of a long stream, with borders inside the pieces."""
    lens = [3000, 1, 0, 2600, 777]
    a = ssm_inputs(21, sum(lens), 32, 16, 1, FP, len(lens), slow=True)
    y, fin = run_scan(a, lens)
    ry, rf = ssm_ref(a["u"], a["dt"], a["A"], a["B"], a["C"], lens, a["D"], a["z"], a["dt_bias"], True, a["init"])
    ey, ef = scan_bounds(a, lens)
    within(y, ry, ey + U32 * ry.abs(), "y")
    within(fin, rf, ef, "final_state")


def test_scan_sequences_stand_alone():
    """Infinities and NaN in one sequence stay in it, also across the pieces that a long stream is cut into; so does a
    decay of zero and one of everything."""
    lens = [900, 1500, 0, 800]
    a = ssm_inputs(22, sum(lens), 64, 16, 1, FP, len(lens))
    clean = run_scan(a, lens)
    a["u"][1000, 3], a["dt"][1200, 5], a["B"][2399, 0, 2] = float("nan"), float("inf"), float("-inf")
    y, fin = run_scan(a, lens)
    keep = [i for i in range(sum(lens)) if not 900 <= i < 2400]
    assert torch.equal(y[keep], clean[0][keep])
    assert torch.equal(fin[[0, 2, 3]], clean[1][[0, 2, 3]])
    assert torch.isnan(y[1000, 3]) and torch.isfinite(y[999]).all()


def test_scan_nothing_to_do():
    a = ssm_inputs(23, 0, 16, 8, 1, FP, 3)
    y, fin = run_scan(a, [0, 0, 0])
    assert y.shape == (0, 16) and torch.equal(fin.cpu(), a["init"])
    a["init"] = None
    _, fin = run_scan(a, [0, 0, 0])
    assert not fin.any()
    y, fin = run_scan(a, [])
    assert fin.shape == (0, 16, 8)


@pytest.mark.parametrize("io", [BF, FP])
@pytest.mark.parametrize("n,Ch,N,G,gate", [(1, 1, 8, 1, True), (1, 4096, 16, 1, True), (5, 130, 32, 2, False),
                                           (33, 72, 64, 3, True), (3, 1000, 16, 1, True)])
def test_steps_continue_a_prompt(n, Ch, N, G, io, gate):
    """Single-token steps from a prompt's final states against the 64-bit recurrence over all tokens."""
    lens = [3 + i % 4 for i in range(n)]
    T = sum(lens)
    a = ssm_inputs(n + Ch, T, Ch, N, G, io, n, gate=gate)
    k = 2
    new = [ssm_inputs(100 + j, n, Ch, N, G, io, n, gate=gate) for j in range(k)]
    y, state = run_scan(a, lens)
    outs = []
    for s in new:
        outs.append(kda.kda_ssm_step(to(s["u"]), to(s["dt"]), to(a["A"]), to(s["B"]), to(s["C"]), state, D=to(a["D"]),
                                     z=to(s["z"]), dt_bias=to(a["dt_bias"])))
    whole = dict(a)
    cu = cu_of(lens)
    for key in ("u", "dt", "B", "C", "z"):
        if a[key] is None:
            continue
        whole[key] = torch.cat([torch.cat([a[key][cu[i]:cu[i + 1]]] + [s[key][i:i + 1] for s in new]) for i in range(n)])
    ln = [L + k for L in lens]
    ry, rf = ssm_ref(whole["u"], whole["dt"], a["A"], whole["B"], whole["C"], ln, a["D"], whole["z"], a["dt_bias"], True,
                     a["init"])
    ey, ef = scan_bounds(whole, ln)
    c2 = cu_of(ln)
    for j in range(k):
        rows = [c2[i] + lens[i] + j for i in range(n)]
        within(outs[j], ry[rows], ey[rows] + U[io] * (ry[rows].abs() + ey[rows]), f"step {j}")
    within(state, rf, ef, "state")
