"""The differentiable forms together, as a block uses them: norm, projections, convolution, scan; the KDA layer with its
inputs kept in 8 bits; captured training steps."""
import numpy as np
import pytest
import torch

import kimi_delta_attention_16_gb300 as kda
from block_testlib import f64, gen, pack8_ref, randn, ssm_inputs, ssm_ref
from kimi_delta_attention_16_gb300 import synth
from test_gpu_ssm import cu_of

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF, FP = torch.bfloat16, torch.float32


def leaf(t):
    return t.to(DEV).requires_grad_()


def pair(lens):
    host = np.asarray(cu_of(lens), np.int32)
    return torch.from_numpy(host).to(DEV), host


class Mixer:
    """norm -> x, z projections -> conv -> B, C, dt projections -> scan -> output projection, as one block."""

    def __init__(self, seed, d, ch, N, io):
        g = gen(seed)
        self.N, self.ch = N, ch
        s = ssm_inputs(seed, 1, ch, N, 1, io, 1)
        self.p = {"nw": randn(g, d, std=0.1, mean=1.0), "nb": randn(g, d, std=0.1), "w_in": randn(g, 2 * ch, d, std=d ** -0.5),
                  "cw": randn(g, ch, 4, std=0.5), "cb": randn(g, ch, std=0.1),
                  "w_x": randn(g, ch + 2 * N, ch, std=ch ** -0.5), "A": s["A"], "D": s["D"], "dt_bias": s["dt_bias"],
                  "w_out": randn(g, d, ch, std=ch ** -0.5)}

    def gpu(self, x, lens, p, saved):
        n = kda.kda_norm_layer(x, p["nw"], p["nb"], saved=saved)
        xz = n @ p["w_in"].t()
        c = kda.kda_ssm_conv_layer(xz[:, :self.ch], p["cw"], lens, bias=p["cb"], saved=saved)  # strided rows
        h = c @ p["w_x"].t()
        dt, B, C = h[:, :self.ch], h[:, self.ch:self.ch + self.N].unsqueeze(1), h[:, self.ch + self.N:].unsqueeze(1)
        y, fin = kda.kda_ssm_layer(c, dt, p["A"], B, C, lens, D=p["D"], z=xz[:, self.ch:], dt_bias=p["dt_bias"], saved=saved)
        return y @ p["w_out"].t(), fin

    def ref(self, x, lens, p):
        mean = x.mean(1, keepdim=True)
        n = (x - mean) / torch.sqrt(((x - mean) ** 2).mean(1, keepdim=True) + 1e-5) * p["nw"] + p["nb"]
        xz = n @ p["w_in"].t()
        rows, t0 = [], 0
        for L in lens:
            xs = torch.cat([torch.zeros(3, self.ch, dtype=x.dtype), xz[t0:t0 + L, :self.ch]])
            rows.append(p["cb"] + sum(xs[j:j + L] * p["cw"][:, j] for j in range(4)))
            t0 += L
        pre = torch.cat(rows)
        c = pre * torch.sigmoid(pre)
        h = c @ p["w_x"].t()
        y, fin = ssm_ref(c, h[:, :self.ch], p["A"], h[:, self.ch:self.ch + self.N].unsqueeze(1),
                         h[:, self.ch + self.N:].unsqueeze(1), lens, p["D"], xz[:, self.ch:], p["dt_bias"], True, None)
        return y @ p["w_out"].t(), fin


def test_block_gradients_fp32():
    """Every parameter's and the input's gradient of the whole block against autograd in 64 bits.  fp32 with library matrix
    products between (TF32 off): relative to each gradient's norm, 1,000 roundings of 2^-24 in quadrature and a factor 10 of
    amplification along five layers stay below 2e-5."""
    lens = [33, 0, 1, 70]
    m = Mixer(3, 48, 64, 16, FP)
    g = gen(4)
    x, dy = randn(g, sum(lens), 48), randn(g, sum(lens), 48)
    assert not torch.backends.cuda.matmul.allow_tf32
    p = {k: leaf(v) for k, v in m.p.items()}
    xg = leaf(x)
    out, fin = m.gpu(xg, cu_of(lens), p, "io")
    got = torch.autograd.grad((out * dy.to(DEV)).sum() + fin.square().sum(), [xg, *p.values()])
    r = {k: f64(v).requires_grad_() for k, v in m.p.items()}
    xr = f64(x).requires_grad_()
    ro, rf = m.ref(xr, lens, r)
    ref = torch.autograd.grad((ro * f64(dy)).sum() + rf.square().sum(), [xr, *r.values()])
    for name, a, b in zip(["x", *p], got, ref):
        assert (f64(a) - b).norm() <= 2e-5 * b.norm(), name
    assert (f64(out) - ro).norm() <= 2e-5 * ro.norm()


def test_saved_8bit_is_the_gradient_at_the_rounded_inputs():
    """saved="e4m3": the forward is untouched, and the gradients equal the direct call's on the values that the 8-bit
    form stands for, bit by bit."""
    lens = [40, 25]
    a = ssm_inputs(9, 65, 96, 16, 1, BF, 2)
    v = {k: t.to(DEV) for k, t in a.items()}
    dy, dfin = randn(gen(10), 65, 96, dtype=BF).to(DEV), randn(gen(11), 2, 96, 16).to(DEV)
    leaves = {k: t.clone().requires_grad_() for k, t in v.items()}
    args = lambda q: (q["u"], q["dt"], q["A"], q["B"], q["C"])  # noqa: E731
    more = lambda q: dict(D=q["D"], z=q["z"], dt_bias=q["dt_bias"], initial_state=q["init"])  # noqa: E731
    y, fin = kda.kda_ssm_layer(*args(leaves), cu_of(lens), **more(leaves), saved="e4m3")
    y0, fin0 = kda.kda_ssm_scan(*args(v), cu_of(lens), **more(v))
    assert torch.equal(y, y0) and torch.equal(fin, fin0)
    got = torch.autograd.grad([y, fin], list(leaves.values()), [dy, dfin])
    w = dict(v, u=kda.kda_unpack8(*kda.kda_pack8(v["u"])), z=kda.kda_unpack8(*kda.kda_pack8(v["z"])))
    assert torch.equal(w["u"].cpu().double(), pack8_ref(a["u"])[0].to(BF).double())
    ref = kda.kda_ssm_backward(*args(w), cu_of(lens), dy, **more(w), d_final_state=dfin)
    names = dict(u="du", dt="ddt", A="dA", B="dB", C="dC", D="dD", z="dz", dt_bias="ddt_bias", init="dinitial_state")
    for k, t in zip(leaves, got):
        assert torch.equal(t, ref[names[k]]), k

    x, w4, bias = v["u"].clone().requires_grad_(), randn(gen(12), 96, 4).to(DEV).requires_grad_(), leaf(randn(gen(13), 96))
    st = randn(gen(14), 2, 96, 3, dtype=BF).to(DEV).requires_grad_()
    yc = kda.kda_ssm_conv_layer(x, w4, cu_of(lens), bias=bias, conv_state_in=st, saved="e4m3")
    got = torch.autograd.grad(yc, [x, w4, bias, st], dy)
    ref = kda.kda_ssm_conv_backward(w["u"], w4.detach(), cu_of(lens), dy, bias=bias.detach(), conv_state_in=st.detach())
    assert torch.equal(got[0], ref["dx"]) and torch.equal(got[1], ref["dw"]) and torch.equal(got[2], ref["dbias"])
    assert torch.equal(got[3], ref["dconv_state_in"].to(BF))


@pytest.mark.parametrize("gate", [True, False])
@pytest.mark.parametrize("strided", [False, True])
def test_kda_layer_with_inputs_kept_in_8_bits(gate, strided):
    """kda_layer(saved="e4m3"): the same outputs, and the gradients of the layer at the rounded q, k, v and gate."""
    inp = synth.make_prefill("layer_8k", seed=31, device=DEV, lengths=[70, 130], H=2, s0_std=0.02, conv_state=True)
    g = gen(32)
    dy = randn(g, 200, 2, 128, dtype=BF).to(DEV)
    q, k, v = inp.q, inp.k, inp.v
    if strided:
        buf = torch.stack([q, k, v], 1).reshape(200, 6, 128)
        q, k, v = (buf[:, 2 * i:2 * i + 2] for i in range(3))

    def grads(q, k, v, gt, saved):
        ins = [t.detach().requires_grad_() for t in (q, k, v, inp.conv_w, inp.g, inp.beta, inp.rms_w, inp.initial_state)]
        gt = None if gt is None else gt.detach().requires_grad_()
        out, fin = kda.kda_layer(*ins[:6], inp.cu_seqlens, gate=gt, rms_w=ins[6], initial_state=ins[7],
                                 conv_state_in=inp.conv_state_in, saved=saved)
        return out, torch.autograd.grad((out * dy).sum() + fin.sum(), ins + ([gt] if gt is not None else []))

    gt = inp.gate if gate else None
    out8, got = grads(q, k, v, gt, "e4m3")
    out, _ = grads(q, k, v, gt, "io")
    assert torch.equal(out8, out)

    def rounded(t):
        return kda.kda_unpack8(*kda.kda_pack8(t.reshape(200, -1)), dtype=t.dtype).view(t.shape)
    _, ref = grads(rounded(q), rounded(k), rounded(v), None if gt is None else rounded(gt), "io")
    for i, (a, b) in enumerate(zip(got, ref)):
        if i in (3, 5, 6):
            # conv_w, beta and rms_w: kda_backward adds them up with atomics, so the order of at most a few hundred
            # partial sums changes, each by 2^-24 of what is summed: under 1e-5 of the norm with terms of either sign
            assert (a - b).norm() <= 1e-5 * b.norm()
        else:
            assert torch.equal(a, b), i


def test_captured_training_step_and_the_refusal():
    """A training step of the layers captured into a graph and replayed on new inputs gives the eager step's gradients.
    While an eager graph of the same leaves lives, the capture is refused before anything is recorded."""
    lens = pair([50, 14])
    a = ssm_inputs(15, 64, 64, 16, 1, BF, 2)
    v = {k: leaf(t) for k, t in a.items()}
    w, b = leaf(randn(gen(16), 64)), leaf(randn(gen(17), 64))
    cw, cb = leaf(randn(gen(18), 64, 4)), leaf(randn(gen(19), 64))
    dy = randn(gen(20), 64, 64, dtype=BF).to(DEV)
    leaves = [*v.values(), w, b, cw, cb]

    def step(saved):
        x = kda.kda_norm_layer(v["u"], w, b, saved=saved)
        x = kda.kda_ssm_conv_layer(x, cw, lens, bias=cb, saved=saved)
        y, fin = kda.kda_ssm_layer(x, v["dt"], v["A"], v["B"], v["C"], lens, D=v["D"], z=v["z"], dt_bias=v["dt_bias"],
                                   initial_state=v["init"], saved=saved)
        return y

    for saved in ("io", "e4m3"):
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            torch.autograd.grad(step(saved), leaves, dy)
        torch.cuda.current_stream().wait_stream(side)
        alive = step(saved)
        graph = torch.cuda.CUDAGraph()
        with pytest.raises(RuntimeError, match="alive"):
            with torch.cuda.graph(graph, stream=side):
                step(saved)
        del alive
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            cap = torch.autograd.grad(step(saved), leaves, dy)
        with torch.no_grad():
            v["u"].mul_(0.5)
            w.add_(0.25)
        graph.replay()
        torch.cuda.synchronize()
        ref = torch.autograd.grad(step(saved), leaves, dy)
        assert all(torch.equal(x, y) for x, y in zip(cap, ref))


def test_two_captured_graphs_keep_their_own_workspaces():
    """Two graphs over different inputs, replayed in turn and then at the same time on two streams."""
    cases = []
    for seed, T in ((40, 900), (41, 700)):
        a = {k: t.to(DEV) for k, t in ssm_inputs(seed, T, 64, 16, 1, BF, 1).items()}
        dy, lens = randn(gen(seed), T, 64, dtype=BF).to(DEV), pair([T])

        def run(a=a, dy=dy, lens=lens):
            ins = (a["u"], a["dt"], a["A"], a["B"], a["C"], lens)
            more = dict(D=a["D"], z=a["z"], dt_bias=a["dt_bias"], initial_state=a["init"])
            y, fin = kda.kda_ssm_scan(*ins, **more)
            return [y, fin, *kda.kda_ssm_backward(*ins, dy, **more).values()]
        want = run()
        graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.graph(graph, stream=side):
            out = run()
        cases.append((graph, out, want, torch.cuda.Stream(), run))  # run: a graph's inputs have to outlive it
    for graph, out, want, *_ in cases + cases:
        for t in out:
            t.zero_()
        graph.replay()
        assert all(torch.equal(x, y) for x, y in zip(out, want))
    torch.cuda.synchronize()
    for _ in range(20):
        for graph, _, _, s, _ in cases:
            with torch.cuda.stream(s):
                graph.replay()
    torch.cuda.synchronize()
    for _, out, want, *_ in cases:
        assert all(torch.equal(x, y) for x, y in zip(out, want))


def test_calls_on_another_stream():
    """stream=: outputs and workspace belong to that stream; the results are the same."""
    a = {k: t.to(DEV) for k, t in ssm_inputs(50, 900, 64, 16, 1, BF, 1).items()}
    ins = (a["u"], a["dt"], a["A"], a["B"], a["C"], pair([900]))
    more = dict(D=a["D"], z=a["z"], dt_bias=a["dt_bias"], initial_state=a["init"])
    dy = randn(gen(51), 900, 64, dtype=BF).to(DEV)
    y, fin = kda.kda_ssm_scan(*ins, **more)
    g = kda.kda_ssm_backward(*ins, dy, **more)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    for st in (s, s.cuda_stream):
        y2, fin2 = kda.kda_ssm_scan(*ins, **more, stream=st)
        junk = [torch.full((1 << 20,), float("nan"), device=DEV) for _ in range(8)]  # takes freed memory of this stream
        g2 = kda.kda_ssm_backward(*ins, dy, **more, stream=st)
        torch.cuda.synchronize()
        del junk
        assert torch.equal(y, y2) and torch.equal(fin, fin2) and all(torch.equal(g[k], g2[k]) for k in g)
