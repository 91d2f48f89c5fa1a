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


# ------------------------------------------------------------------ gradients of the scan
GRADS = {"u": "du", "dt": "ddt", "A": "dA", "B": "dB", "C": "dC", "D": "dD", "z": "dz", "dt_bias": "ddt_bias",
         "init": "dinitial_state"}


def ref_grads(a, lens, dy, dfin, softplus=True):
    """The formula's gradients, by autograd over the 64-bit recurrence."""
    leaves = {k: f64(t).requires_grad_() for k, t in a.items() if t is not None}
    v = {k: leaves.get(k) for k in a}
    y, fin = ssm_ref(v["u"], v["dt"], v["A"], v["B"], v["C"], lens, v["D"], v["z"], v["dt_bias"], softplus, v["init"])
    loss = (y * f64(dy)).sum() + (0 if dfin is None else (fin * f64(dfin)).sum())
    got = torch.autograd.grad(loss, list(leaves.values()), allow_unused=True)
    return {GRADS[k]: (torch.zeros_like(leaves[k]) if g is None else g) for k, g in zip(leaves, got)}


def run_backward(a, lens, dy, dfin, how="dense", **kw):
    v = {k: (rows_in(t, how) if k in ("u", "dt", "z") and t is not None else to(t)) for k, t in a.items()}
    return kda.kda_ssm_backward(v["u"], v["dt"], v["A"], v["B"], v["C"], cu_of(lens), rows_in(dy, how), D=v["D"],
                                z=v["z"], dt_bias=v["dt_bias"], initial_state=v["init"], d_final_state=to(dfin), **kw)


def grad_bounds(a, lens, dy, dfin, softplus=True):
    """Bounds of every gradient: the gradients of the same scan on magnitudes (all terms positive, nothing cancels) times
    a relative error.  Every factor of a term carries at most 60 units of the last place (two step sizes, an exponential,
    the gate and its slope, up to eight products), a state's and its gradient's memory adds 4 units per token of it, and a
    sum over K terms K units.  The exponent delta A comes with 13 units (10 of delta, 3 of A log2 e and the product), and an
    error d of an exponent E is a relative error d E of e^E: a term that has passed k decays of exponent x each has 13 k x
    units, and weighted by the terms' own size e^(-k x) the mean of k x is at most 1 beyond the decay that the term itself
    carries, for the state and for its gradient: 13 (2 max|delta A| + 2) units."""
    mag = {k: (None if t is None else f64(t).abs()) for k, t in a.items()}
    x = f64(a["dt"]) + (0 if a["dt_bias"] is None else f64(a["dt_bias"]))
    delta = (torch.logaddexp(x, torch.zeros_like(x)) if softplus else x).abs()
    T, Ch = delta.shape
    G, N = a["B"].shape[1:]
    u, B, C = (mag[k] for k in ("u", "B", "C"))
    A = f64(a["A"])
    wide = lambda r: r.unsqueeze(1).expand(G, Ch // G, N).reshape(Ch, N)  # noqa: E731
    sz = dsz = torch.ones(T, Ch, dtype=torch.float64)
    if a["z"] is not None:
        z = f64(a["z"])
        sg = torch.sigmoid(z)
        sz, dsz = (z * sg).abs(), (sg * (1 + z.abs()))
    g = f64(dy).abs() * sz
    skip = torch.zeros(Ch, dtype=torch.float64) if a["D"] is None else f64(a["D"]).abs()
    k = {n: torch.zeros_like(t) for n, t in (("du", u), ("ddt", u), ("dz", u), ("dB", B), ("dC", C), ("dA", A))}
    k["dD"], k["ddt_bias"] = torch.zeros(Ch, dtype=torch.float64), torch.zeros(Ch, dtype=torch.float64)
    k["dinitial_state"] = torch.zeros(len(lens), Ch, N, dtype=torch.float64)
    # relative error of states and their gradients: per token of memory, at most the memory's length
    mem = 0.0
    t0 = 0
    for i, L in enumerate(lens):
        h = torch.zeros(Ch, N, dtype=torch.float64) if a["init"] is None else mag["init"][i]
        hist = []
        for t in range(t0, t0 + L):
            hist.append(h)
            h = torch.exp(delta[t].unsqueeze(1) * A) * h + (delta[t] * u[t]).unsqueeze(1) * wide(B[t])
        hist.append(h)
        q = torch.zeros(Ch, N, dtype=torch.float64) if dfin is None else f64(dfin)[i].abs()
        for t in range(t0 + L - 1, t0 - 1, -1):
            h, before = hist[t - t0 + 1], hist[t - t0]
            d = delta[t].unsqueeze(1)
            dec = torch.exp(d * A)
            lam = q + g[t].unsqueeze(1) * wide(C[t])
            k["dC"][t] += (g[t].unsqueeze(1) * h).view(G, Ch // G, N).sum(1)
            k["dB"][t] += (lam * d * u[t].unsqueeze(1)).view(G, Ch // G, N).sum(1)
            s1 = (lam * wide(B[t])).sum(1)
            w = lam * dec * before
            k["dA"] += w * d
            k["du"][t] = delta[t] * s1 + skip * g[t]
            slope = torch.sigmoid(x[t]) if softplus else 1.0
            k["ddt"][t] = (u[t] * s1 + (w * A.abs()).sum(1)) * slope
            k["dz"][t] = f64(dy)[t].abs() * ((wide(C[t]) * h).sum(1) + skip * u[t]) * dsz[t]
            q = dec * lam
        if L == 0 and dfin is not None:
            q = f64(dfin)[i].abs()
        k["dinitial_state"][i] = q
        t0 += L
    k["dD"], k["ddt_bias"] = (g * u).sum(0), k["ddt"].sum(0)
    steps = min(max(lens), 4000)
    rel = (60 + 2 * x.abs().max().item() * 4) * U32 + 4 * steps * U32 * 0.25 * 2
    rel += 13 * U32 * (2 * (delta.unsqueeze(2) * A).abs().max().item() + 2)
    return {n: v * (rel + (Ch if n in ("dB", "dC") else T if n in ("dA", "dD", "ddt_bias") else N) * U32) + 1e-30
            for n, v in k.items()}


BWD_LENS = [[1], [2, 3], [4, 8, 12], [0, 16, 0, 33, 1, 0, 1, 1, 6], [131], [90, 3, 260]]


@pytest.mark.parametrize("lens", BWD_LENS)
@pytest.mark.parametrize("Ch,N,G,how,io", [
    (64, 16, 1, "dense", BF), (128, 16, 1, "dense", FP), (40, 8, 2, "odd", BF), (1, 16, 1, "dense", FP),
    (96, 32, 3, "strided", BF), (130, 64, 2, "dense", FP), (300, 8, 1, "odd", FP), (65, 64, 1, "dense", BF)])
def test_scan_gradients(lens, Ch, N, G, how, io):
    T, n = sum(lens), len(lens)
    a = ssm_inputs(T + Ch + N, T, Ch, N, G, io, n, gate=Ch != 40, skip=Ch != 96, state=Ch != 300, bias=Ch != 65)
    g = gen(T)
    dy, dfin = randn(g, T, Ch, dtype=io), (randn(g, n, Ch, N) if Ch != 130 else None)
    got = run_backward(a, lens, dy, dfin, how)
    ref, tol = ref_grads(a, lens, dy, dfin), grad_bounds(a, lens, dy, dfin)
    assert set(got) == set(ref)
    for name, r in ref.items():
        u = U[io] if name in ("du", "ddt", "dz", "dB", "dC") else 0.0
        within(got[name], r, tol[name] + u * (r.abs() + tol[name]), name)


@pytest.mark.parametrize("lens", [[1500], [700, 0, 1, 900, 64]])
@pytest.mark.parametrize("N,G", [(16, 1), (32, 2)])
def test_scan_gradients_over_pieces(lens, N, G):
    T, n, Ch = sum(lens), len(lens), 48
    a = ssm_inputs(T + N, T, Ch, N, G, FP, n, slow=True)
    g = gen(T)
    dy, dfin = randn(g, T, Ch), randn(g, n, Ch, N)
    got = run_backward(a, lens, dy, dfin)
    ref, tol = ref_grads(a, lens, dy, dfin), grad_bounds(a, lens, dy, dfin)
    for name, r in ref.items():
        within(got[name], r, tol[name] + U32 * r.abs(), name)
    again = run_backward(a, lens, dy, dfin, check_cu_on_host=False)
    assert all(torch.equal(got[k], again[k]) for k in got)  # fixed order of the sums


def test_scan_gradients_against_differences():
    """Central differences of the GPU scan itself, along random directions (fp32: a step of 2^-6 leaves a truncation error
    of h^2 times the third derivative, and a rounding error of 2^-24 |loss terms| / h)."""
    lens = [37, 20]
    a = ssm_inputs(77, 57, 32, 16, 1, FP, 2)
    g = gen(78)
    dy, dfin = randn(g, 57, 32), randn(g, 2, 32, 16)
    got = run_backward(a, lens, dy, dfin)
    step = 2.0 ** -6
    for k, name in GRADS.items():
        v = randn(g, *a[k].shape)
        v /= v.norm()
        if k in ("A", "dt"):
            v *= 0.5

        def loss(sign):
            b = dict(a)
            b[k] = a[k] + sign * step * v
            y, fin = ssm_ref(b["u"], b["dt"], b["A"], b["B"], b["C"], lens, b["D"], b["z"], b["dt_bias"], True, b["init"])
            yg, fg = run_scan(b, lens)
            return (yg.cpu().double() * f64(dy)).sum() + (fg.cpu().double() * f64(dfin)).sum(), (y * f64(dy)).abs().sum()

        (hi, mag), (lo, _) = loss(1), loss(-1)
        want = ((hi - lo) / (2 * step)).item()
        have = (got[name].cpu().double() * v).sum().item()
        scale = got[name].cpu().double().norm().item()
        assert abs(want - have) <= 0.02 * scale + 64 * U32 * float(mag) / step, (name, want, have, scale)


def test_scan_gradients_nothing_to_do():
    a = ssm_inputs(23, 0, 16, 8, 1, FP, 2)
    dfin = randn(gen(1), 2, 16, 8)
    got = run_backward(a, [0, 0], torch.empty(0, 16), dfin)
    assert torch.equal(got["dinitial_state"].cpu(), dfin)
    assert not got["dA"].any() and not got["dD"].any() and not got["ddt_bias"].any()


@pytest.mark.parametrize("bad", [[0, 50, 20, 64], [3, 10, 30, 64], [0, 10, 90, 64], [0, 10, 30, 60], [0, -5, 30, 64]])
def test_inconsistent_device_cu_seqlens_is_reported(bad):
    """A device-only cu_seqlens that does not partition the tokens is flagged through d_status; every index stays in
    range (sequence numbers and ranges are clamped), so the call ends and the next one is right."""
    import numpy as np
    from kimi_delta_attention_16_gb300 import _lib
    a = ssm_inputs(61, 64, 64, 16, 1, FP, 3)
    v = {k: to(t) for k, t in a.items()}
    cu = (torch.tensor(bad, dtype=torch.int32, device=DEV), np.asarray([0, 10, 30, 64], np.int32))
    kw = dict(check_cu_on_host=False)
    x, w, dy = v["u"], randn(gen(62), 64, 4).to(DEV), randn(gen(63), 64, 64).to(DEV)
    ins, more = (v["u"], v["dt"], v["A"], v["B"], v["C"]), dict(D=v["D"], z=v["z"], dt_bias=v["dt_bias"], initial_state=v["init"])
    calls = [lambda s: kda.kda_ssm_conv(x, w, cu, output_conv_state=True, d_status=s, **kw),
             lambda s: kda.kda_ssm_conv_backward(x, w, cu, dy, d_status=s, **kw),
             lambda s: kda.kda_ssm_scan(*ins, cu, d_status=s, **more, **kw),
             lambda s: kda.kda_ssm_backward(*ins, cu, dy, d_status=s, **more, **kw)]
    for f in calls:
        status = torch.zeros(1, dtype=torch.int32, device=DEV)
        f(status)
        assert status.item() == _lib.KDA_ERR_DEVICE_ARG
    y, _ = run_scan(a, [10, 20, 34])
    ry, _ = ssm_ref(a["u"], a["dt"], a["A"], a["B"], a["C"], [10, 20, 34], a["D"], a["z"], a["dt_bias"], True, a["init"])
    ey, _ = scan_bounds(a, [10, 20, 34])
    within(y, ry, ey + U32 * ry.abs(), "y")


def test_large_offsets():
    """Rows whose offsets pass 32 bits: strided views with a row stride of 2^26 + 8 elements (bf16, 40 rows: 5 GB)."""
    stride, T, C = (1 << 26) + 8, 40, 64
    buf = torch.empty(stride * T, dtype=BF, device=DEV)
    a = ssm_inputs(71, T, C, 16, 1, BF, 2)

    def far(t, off):
        view = torch.as_strided(buf, (T, C), (stride, 1), off)
        view.copy_(t.to(DEV))
        return view
    u, dt, z, x = far(a["u"], 0), far(a["dt"], 64), far(a["z"], 128), far(a["u"] * 2, 192)
    lens = [30, 10]
    rest = (to(a["A"]), to(a["B"]), to(a["C"]))
    more = dict(D=to(a["D"]), dt_bias=to(a["dt_bias"]), initial_state=to(a["init"]))
    y, fin = kda.kda_ssm_scan(u, dt, *rest, cu_of(lens), z=z, **more)
    y0, fin0 = kda.kda_ssm_scan(to(a["u"]), to(a["dt"]), *rest, cu_of(lens), z=to(a["z"]), **more)
    assert torch.equal(y, y0) and torch.equal(fin, fin0)
    st, st0 = fin.repeat(20, 1, 1).contiguous(), fin.repeat(20, 1, 1).contiguous()
    y = kda.kda_ssm_step(u, dt, *rest, st, z=z, D=more["D"], dt_bias=more["dt_bias"])
    y0 = kda.kda_ssm_step(to(a["u"]), to(a["dt"]), *rest, st0, z=to(a["z"]), D=more["D"], dt_bias=more["dt_bias"])
    assert torch.equal(y, y0) and torch.equal(st, st0)
    w = randn(gen(72), C, 4).to(DEV)
    assert torch.equal(kda.kda_ssm_conv(x, w, cu_of(lens)), kda.kda_ssm_conv(to(a["u"] * 2), w, cu_of(lens)))
    n, ns = kda.kda_layer_norm(x, return_stats=True)
    m, ms = kda.kda_layer_norm(to(a["u"] * 2), return_stats=True)
    assert torch.equal(n, m) and torch.equal(ns, ms)
    g, g0 = kda.kda_layer_norm_backward(u, x, ns), kda.kda_layer_norm_backward(to(a["u"]), to(a["u"] * 2), ms)
    assert all(torch.equal(g[k], g0[k]) for k in g)
    c, c0 = kda.kda_pack8(x), kda.kda_pack8(to(a["u"] * 2))
    assert torch.equal(c[0], c0[0]) and torch.equal(c[1], c0[1])
    out = torch.as_strided(buf, (T, C), (stride, 1), 256)
    assert torch.equal(kda.kda_unpack8(*c, out=out), kda.kda_unpack8(*c))


def test_inputs_of_a_call_on_another_stream_are_marked(monkeypatch):
    """The allocator is told that the other stream reads the inputs, cu_seqlens among them (a list's device copy
    is made on that stream itself)."""
    a = ssm_inputs(5, 32, 16, 16, 1, FP, 1)
    cu = torch.tensor([0, 32], dtype=torch.int32)
    pair = (cu.to(DEV), cu.numpy())
    marked = []
    mark = torch.Tensor.record_stream
    monkeypatch.setattr(torch.Tensor, "record_stream", lambda t, s: (marked.append(t.data_ptr()), mark(t, s))[1])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    w = torch.zeros(16, 4, device=DEV)
    dev = {k: v.to(DEV) if isinstance(v, torch.Tensor) else v for k, v in a.items()}
    s.wait_stream(torch.cuda.current_stream())
    for call in (lambda: kda.kda_ssm_conv(dev["u"], w, pair, stream=s),
                 lambda: kda.kda_ssm_conv_backward(dev["u"], w, pair, dev["u"], stream=s),
                 lambda: kda.kda_ssm_scan(dev["u"], dev["dt"], dev["A"], dev["B"], dev["C"], pair, stream=s),
                 lambda: kda.kda_ssm_backward(dev["u"], dev["dt"], dev["A"], dev["B"], dev["C"], pair, dev["u"], stream=s)):
        marked.clear()
        call()
        assert pair[0].data_ptr() in marked and dev["u"].data_ptr() in marked
    s.synchronize()


SHORT = [37, 5, 90, 1, 0, 64, 8, 200, 3, 120, 16, 31, 64, 64, 7, 400, 2, 128, 129, 63, 1]


@pytest.mark.parametrize("how", ["dense", "odd"])
@pytest.mark.parametrize("Ch,N,G,io", [(48, 16, 1, FP), (26, 32, 2, BF), (40, 8, 1, BF), (20, 64, 2, FP)])
def test_short_sequences_over_pieces(Ch, N, G, io, how):
    """Pieces that hold several sequences: only the last that starts in one leaves a state to the next, and only the
    first that ends in one sends a gradient back.  Initial and final states of all of them take part."""
    T, n = sum(SHORT), len(SHORT)
    a = ssm_inputs(T + Ch, T, Ch, N, G, io, n, slow=True)
    y, fin = run_scan(a, SHORT, how)
    ry, rf = ssm_ref(a["u"], a["dt"], a["A"], a["B"], a["C"], SHORT, a["D"], a["z"], a["dt_bias"], True, a["init"])
    ey, ef = scan_bounds(a, SHORT)
    within(y, ry, ey + U[io] * (ry.abs() + ey), "y")
    within(fin, rf, ef, "final_state")
    g = gen(T + 1)
    dy, dfin = randn(g, T, Ch, dtype=io), randn(g, n, Ch, N)
    got = run_backward(a, SHORT, dy, dfin, how)
    ref, tol = ref_grads(a, SHORT, dy, dfin), grad_bounds(a, SHORT, dy, dfin)
    for name, r in ref.items():
        u = U[io] if name in ("du", "ddt", "dz", "dB", "dC") else 0.0
        within(got[name], r, tol[name] + u * (r.abs() + tol[name]) + U32 * r.abs(), name)
