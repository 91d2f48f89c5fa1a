"""The operators around a hybrid block's second token mixer, as one measured set: layer norm with its gradient,
activation checkpoints in 8 bits, and a selective state space scan with its short causal convolution.

Each case is one pass through one operator.  ``run`` computes it in plain torch operations (fp32, rounded once at
the end) or, with ``own`` set, through the package's entry points; ``exact`` computes it in 64 bits, token by token.
"""
import math

import numpy as np
import torch

own = False

_DT = {"bf16": torch.bfloat16, "fp32": torch.float32}
EPS = 1e-5


# ------------------------------------------------------------------ cases
def listed():
    return [
        # the norm in front of one decode step of 256 sequences, at the backbone's width
        dict(name="norm_decode_256", op="norm", rows=256, width=7168, io="bf16"),
        # training: forward and backward of that norm over one 8,192-token sequence
        dict(name="norm_train_8k", op="norm_train", rows=8192, width=7168, io="bf16", saved="io"),
        # an odd width (scalar tail everywhere), a ragged number of rows, fp32
        dict(name="norm_train_odd_fp32", op="norm_train", rows=1237, width=1001, io="fp32", saved="io"),
        # the same training step with the norm's input kept in 8 bits for the backward pass
        dict(name="norm_train_8bit", op="norm_train", rows=8192, width=7168, io="bf16", saved="e4m3"),
        # one 8,192-token activation of 96 heads of 128 packed for the backward pass and read back
        dict(name="pack8_8k", op="pack8", rows=8192, width=12288, io="bf16"),
        # the short convolution in training, packed sequences of unequal length
        dict(name="conv_train_varlen", op="conv_train", lens="2048,517,3001,64,1,1500,1061", ch=8192, io="bf16",
             state=False),
        # the short convolution of one decode step of 256 sequences
        dict(name="conv_step_256", op="conv_step", batch=256, ch=12288, io="bf16"),
        # one 8,192-token prompt through the scan
        dict(name="scan_prompt_8k", op="scan", lens="8192", ch=12288, n=16, groups=1, io="bf16", state=False, gate=True),
        # packed prompts that continue from states, few channels (long chains, little parallelism), fp32, 4 groups
        dict(name="scan_varlen_fp32", op="scan", lens="700,1,2048,4096,33,1201", ch=1536, n=32, groups=4, io="fp32",
             state=True, gate=True),
        # decode: one token for each of 256 sequences
        dict(name="step_256", op="step", batch=256, ch=12288, n=16, groups=1, io="bf16", gate=True),
        # decode of a single sequence, where latency counts
        dict(name="step_1", op="step", batch=1, ch=4096, n=16, groups=1, io="bf16", gate=True),
        # training: forward and backward of the scan over one 4,096-token sequence
        dict(name="scan_train_4k", op="scan_train", lens="4096", ch=4096, n=16, groups=1, io="bf16", state=False,
             gate=True),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _lens(rng, total):
    """One to eight sequences of `total` tokens in all, unequal, now and then an empty one."""
    cuts = sorted(rng.randint(0, total) for _ in range(rng.choice([0, 0, 1, 3, 7])))
    return ",".join(str(b - a) for a, b in zip([0] + cuts, cuts + [total]))


def draw(rng):
    io = rng.choice(["bf16", "bf16", "fp32"])
    op = rng.choice(["norm", "norm_train", "pack8", "conv_train", "conv_step", "scan", "scan", "step", "scan_train"])
    if op in ("norm", "norm_train", "pack8"):
        width = _log_int(rng, 64, 16384)
        rows = _log_int(rng, 1, min(32768, (32 << 20) // width))
        c = dict(op=op, rows=rows, width=width, io=io)
        if op == "norm_train":
            c["saved"] = rng.choice(["io", "e4m3"])
        return c
    n = rng.choice([8, 16, 16, 16, 32, 64])
    groups = rng.choice([1, 1, 2, 4])
    ch = 8 * groups * _log_int(rng, 8, 12288 // (8 * groups))
    if op == "conv_step":
        return dict(op=op, batch=_log_int(rng, 1, 512), ch=ch, io=io)
    if op == "step":
        return dict(op=op, batch=_log_int(rng, 1, min(512, (1 << 26) // (ch * n))), ch=ch, n=n, groups=groups, io=io,
                    gate=rng.random() < 0.7)
    if op == "conv_train":
        return dict(op=op, lens=_lens(rng, _log_int(rng, 1, min(16384, (1 << 25) // ch))), ch=ch, io=io,
                    state=rng.random() < 0.5)
    most = (1 << 28) if op == "scan" else (1 << 27)
    total = _log_int(rng, 1, max(2, min(16384, most // (ch * n))))
    return dict(op=op, lens=_lens(rng, total), ch=ch, n=n, groups=groups, io=io, state=rng.random() < 0.5,
                gate=rng.random() < 0.7)


# ------------------------------------------------------------------ inputs
class _Maker:
    def __init__(self, seed):
        self.g = torch.Generator(device="cuda")
        self.g.manual_seed(int(seed))

    def normal(self, *shape, std=1.0, mean=0.0, dtype=torch.float32):
        return (torch.randn(*shape, generator=self.g, device="cuda") * std + mean).to(dtype)

    def uniform(self, *shape, lo=0.0, hi=1.0, dtype=torch.float32):
        return (torch.rand(*shape, generator=self.g, device="cuda") * (hi - lo) + lo).to(dtype)


def _cu(lens):
    host = np.zeros(len(lens) + 1, np.int32)
    host[1:] = np.cumsum(np.asarray(lens, np.int64))
    return torch.from_numpy(host).cuda(), host


def prepare(case, seed):
    m, op, io = _Maker(seed), case["op"], _DT[case["io"]]
    s = {"op": op, "io": io}
    if op in ("norm", "norm_train"):
        M, W = case["rows"], case["width"]
        # a residual stream: a few channels much larger than the others
        s["x"] = (m.normal(M, W) * torch.exp(m.normal(W, std=0.7)) + m.normal(W, std=0.3)).to(io)
        s["weight"], s["bias"] = m.normal(W, std=0.1, mean=1.0), m.normal(W, std=0.1)
        if op == "norm_train":
            s["dy"], s["saved"] = m.normal(M, W, dtype=io), case["saved"]
        return s
    if op == "pack8":
        s["x"] = (m.normal(case["rows"], case["width"]) * torch.exp(m.normal(case["width"]))).to(io)
        return s
    Ch = case["ch"]
    if op in ("conv_train", "conv_step"):
        s["w"], s["bias"] = m.normal(Ch, 4, std=0.5), m.normal(Ch, std=0.1)
        if op == "conv_step":
            s["x"] = m.normal(case["batch"], Ch, dtype=io)
            s["conv_state"] = m.normal(case["batch"], Ch, 3, dtype=io)
            return s
        lens = [int(v) for v in case["lens"].split(",")]
        s["cu"], T = _cu(lens), sum(lens)
        s["x"], s["dy"] = m.normal(T, Ch, dtype=io), m.normal(T, Ch, dtype=io)
        s["conv_state"] = m.normal(len(lens), Ch, 3, dtype=io) if case["state"] else None
        return s
    N, G = case["n"], case["groups"]
    if op == "step":
        rows = case["batch"]
        s["state"] = m.normal(rows, Ch, N, std=0.1)
    else:
        lens = [int(v) for v in case["lens"].split(",")]
        s["cu"], rows = _cu(lens), sum(lens)
        s["full"] = torch.tensor([i for i, v in enumerate(lens) if v], device="cuda")  # the sequences that are not empty
        s["state"] = m.normal(len(lens), Ch, N, std=0.1) if case["state"] else None
    s["u"] = torch.nn.functional.silu(m.normal(rows, Ch)).to(io)
    s["dt"] = m.normal(rows, Ch, std=0.5, dtype=io)
    # step sizes log-uniform in [1e-3, 1e-1] through the softplus; decay rates 1..N per channel, as trained ones spread
    step = torch.exp(m.uniform(Ch, lo=math.log(1e-3), hi=math.log(1e-1)))
    s["dt_bias"] = step + torch.log(-torch.expm1(-step))
    s["A"] = -torch.arange(1, N + 1, device="cuda", dtype=torch.float32) * torch.exp(m.normal(Ch, N, std=0.1))
    s["B"], s["C"] = m.normal(rows, G, N, dtype=io), m.normal(rows, G, N, dtype=io)
    s["D"] = m.normal(Ch, std=0.1, mean=1.0)
    s["z"] = m.normal(rows, Ch, dtype=io) if case["gate"] else None
    if op == "scan_train":
        s["dy"] = m.normal(rows, Ch, dtype=io)
    return s


# ------------------------------------------------------------------ the plain forms
def _pow2(e):
    """2^e in fp32 for whole e in [-126, 127]."""
    return ((e + 127) << 23).to(torch.int32).view(torch.float32)


def _blocks(x):
    """fp32 rows padded with zeros to whole blocks of 32: [M, blocks, 32]."""
    x = torch.nn.functional.pad(x.float(), (0, -x.shape[1] % 32))
    return x.view(x.shape[0], -1, 32)


def _plain_pack8(x):
    """(x as its 8-bit form stands for it, fp32; scale bytes): e4m3 codes in blocks of 32 under one power of two, the
    smallest that brings the block's largest magnitude to at most 448."""
    v = _blocks(x)
    top = v.abs().amax(2)
    frac, e = torch.frexp(top)
    e = torch.where(top > 0, e - 9 + (frac > 0.875), -126).clamp(-126, 127)
    codes = (v * _pow2(-e).unsqueeze(2)).to(torch.float8_e4m3fn)
    back = (codes.float() * _pow2(e).unsqueeze(2)).view(x.shape[0], -1)[:, :x.shape[1]]
    return back, (e + 127).to(torch.uint8)


def _plain_norm(s):
    x, io = s["x"].float(), s["io"]
    mean = x.mean(1, keepdim=True)
    rstd = torch.rsqrt((x - mean).square().mean(1, keepdim=True) + EPS)
    y = ((x - mean) * rstd * s["weight"] + s["bias"]).to(io)
    if s["op"] == "norm":
        return y
    if s["saved"] == "e4m3":
        x = _plain_pack8(s["x"])[0].to(io).float()
    xh, dy = (x - mean) * rstd, s["dy"].float()
    p = dy * s["weight"]
    dx = rstd * (p - p.mean(1, keepdim=True) - xh * (p * xh).mean(1, keepdim=True))
    return {"y": y, "dx": dx.to(io), "dweight": (dy * xh).sum(0), "dbias": dy.sum(0)}


def _taps(x, cu, state):
    """x[t-3], x[t-2], x[t-1], x[t] of each token's own sequence, [4, T, C] fp32; the places before a start come from
    `state` or are zero."""
    T, dev = x.shape[0], x.device
    t = torch.arange(T, device=dev)
    seq = torch.searchsorted(cu, t, right=True) - 1
    pos = t - cu[seq]
    src = t.view(1, -1) + torch.arange(-3, 1, device=dev).view(-1, 1)
    lag = pos.view(1, -1) + torch.arange(-3, 1, device=dev).view(-1, 1)
    inside = (lag >= 0).unsqueeze(2)
    taps = torch.where(inside, x.float()[src.clamp(min=0)], torch.zeros((), device=dev))
    if state is not None:
        taps = torch.where(inside, taps, state.float()[seq.view(1, -1), :, (lag + 3).clamp(0, 2)])
    return taps, seq, src, lag


def _plain_conv_train(s):
    x, cu, st, io = s["x"], s["cu"][0].long(), s["conv_state"], s["io"]
    N, Ch = cu.shape[0] - 1, x.shape[1]
    taps, seq, src, lag = _taps(x, cu, st)
    pre = (taps * s["w"].t().unsqueeze(1)).sum(0) + s["bias"]
    sg = torch.sigmoid(pre)
    y = (pre * sg).to(io)
    dpre = s["dy"].float() * (sg * (1 + pre * (1 - sg)))
    dw = (taps * dpre).sum(1).t().contiguous()
    back = dpre * s["w"].t().unsqueeze(1)
    dx = torch.zeros_like(dpre)
    for j in range(4):
        dx.index_add_(0, src[j].clamp(min=0), torch.where((lag[j] >= 0).unsqueeze(1), back[j], torch.zeros((), device=x.device)))
    # the last three raw values of every sequence, the incoming ones among them where it is shorter
    at = cu[1:].unsqueeze(1) + torch.arange(-3, 0, device=x.device)
    lag_end = at - cu[:-1].unsqueeze(1)
    rows = x[at.clamp(0, max(0, x.shape[0] - 1))]
    keep = (lag_end >= 0).unsqueeze(2)
    old = torch.zeros(N, 3, Ch, device=x.device, dtype=io) if st is None else st.transpose(1, 2).gather(
        1, (lag_end + 3).clamp(0, 2).unsqueeze(2).expand(N, 3, Ch))
    out = {"y": y, "dx": dx.to(io), "dw": dw, "dbias": dpre.sum(0),
           "conv_state": torch.where(keep, rows, old).transpose(1, 2).contiguous()}
    if st is not None:
        flat = torch.zeros(N * 3, Ch, device=x.device)
        for j in range(3):
            flat.index_add_(0, seq * 3 + (lag[j] + 3).clamp(0, 2), torch.where((lag[j] < 0).unsqueeze(1), back[j], torch.zeros((), device=x.device)))
        out["dconv_state_in"] = flat.view(N, 3, Ch).transpose(1, 2).contiguous()
    return out


def _plain_conv_step(s):
    st = s["conv_state"]
    win = torch.cat([st, s["x"].unsqueeze(2)], 2)
    pre = (win.float() * s["w"]).sum(2) + s["bias"]
    st.copy_(win[:, :, 1:].clone())
    return {"y": (pre * torch.sigmoid(pre)).to(s["io"]), "conv_state": st}


def _softplus(x):
    return torch.where(x > 20, x, torch.log1p(torch.exp(x.clamp(max=20))))


def _per_channel(b, ch):
    """[T, G, N] -> [T, ch, N] fp32: every channel of a group reads the group's row."""
    T, G, N = b.shape
    return b.float().unsqueeze(2).expand(T, G, ch // G, N).reshape(T, ch, N)


def _scan(a, b, longest):
    """h_t = a_t h_{t-1} + b_t along dim 0, by doubling."""
    k = 1
    while k < longest:
        b[k:] = b[k:] + a[k:] * b[:-k]
        a[k:] = a[k:] * a[:-k]
        k *= 2
    return b


def _plain_scan(s):
    io, T, Ch = s["io"], *s["u"].shape
    cu, host = s["cu"]
    N = s["A"].shape[1]
    longest = int(np.max(np.diff(host)))
    full = s["full"]
    starts = cu[:-1].long()[full]
    u, x = s["u"].float(), s["dt"].float() + s["dt_bias"]
    delta = _softplus(x)
    Bc, Cc = _per_channel(s["B"], Ch), _per_channel(s["C"], Ch)
    a = torch.exp(delta.unsqueeze(2) * s["A"])
    b = (delta * u).unsqueeze(2) * Bc
    init = s["state"] if s["state"] is not None else torch.zeros(len(host) - 1, Ch, N, device=u.device)
    a0 = a[starts]
    b[starts] += a0 * init[full]
    keep = a.clone() if s["op"] == "scan_train" else None
    a[starts] = 0
    h = _scan(a, b, longest)
    ybar = (Cc * h).sum(2) + s["D"] * u
    z = None if s["z"] is None else s["z"].float()
    sg = None if z is None else torch.sigmoid(z)
    y = (ybar if z is None else ybar * z * sg).to(io)
    final = init.clone()
    final[full] = h[cu[1:].long()[full] - 1]
    if s["op"] == "scan":
        return {"y": y, "final_state": final}
    dy = s["dy"].float()
    out = {"y": y, "final_state": final}
    g = dy
    if z is not None:
        out["dz"] = (dy * ybar * (sg * (1 + z * (1 - sg)))).to(io)
        g = dy * z * sg
    lam = g.unsqueeze(2) * Cc
    r = torch.zeros_like(keep)
    r[:-1] = keep[1:]
    r[cu[1:].long()[full] - 1] = 0
    lam = _scan(r.flip(0), lam.flip(0), longest).flip(0)
    ah = h - (delta * u).unsqueeze(2) * Bc  # a_t h_{t-1}
    G = s["B"].shape[1]
    out["dC"] = (g.unsqueeze(2) * h).view(T, G, Ch // G, N).sum(2).to(io)
    out["dB"] = (lam * (delta * u).unsqueeze(2)).view(T, G, Ch // G, N).sum(2).to(io)
    dbu = (lam * Bc).sum(2)
    out["dA"] = (lam * ah * delta.unsqueeze(2)).sum(0)
    ddelta = dbu * u + (lam * ah * s["A"]).sum(2)
    out["du"] = (dbu * delta + g * s["D"]).to(io)
    out["dD"] = (g * u).sum(0)
    dx = ddelta * torch.sigmoid(x)
    out["ddt"], out["ddt_bias"] = dx.to(io), dx.sum(0)
    if s["state"] is not None:
        dinit = torch.zeros_like(init)
        dinit[full] = a0 * lam[starts]
        out["dinitial_state"] = dinit
    return out


def _plain_step(s):
    u, Ch = s["u"].float(), s["u"].shape[1]
    delta = _softplus(s["dt"].float() + s["dt_bias"])
    h = torch.exp(delta.unsqueeze(2) * s["A"]) * s["state"] + (delta * u).unsqueeze(2) * _per_channel(s["B"], Ch)
    s["state"].copy_(h)
    y = (h * _per_channel(s["C"], Ch)).sum(2) + s["D"] * u
    if s["z"] is not None:
        z = s["z"].float()
        y = y * z * torch.sigmoid(z)
    return {"y": y.to(s["io"]), "state": s["state"]}


def _plain_round(s):
    back, scales = _plain_pack8(s["x"])
    return {"values": back.to(s["io"]), "scales": scales}


_PLAIN = {"norm": _plain_norm, "norm_train": _plain_norm, "pack8": _plain_round, "conv_train": _plain_conv_train,
          "conv_step": _plain_conv_step, "scan": _plain_scan, "scan_train": _plain_scan, "step": _plain_step}


# ------------------------------------------------------------------ the package's operators
def _own(s):
    import kimi_delta_attention_16_gb300 as kda
    op = s["op"]
    if op == "norm":
        return kda.kda_layer_norm(s["x"], s["weight"], s["bias"], eps=EPS)
    if op == "norm_train":
        y, stats = kda.kda_layer_norm(s["x"], s["weight"], s["bias"], eps=EPS, return_stats=True)
        x, scales = kda.kda_pack8(s["x"]) if s["saved"] == "e4m3" else (s["x"], None)
        return {"y": y, **kda.kda_layer_norm_backward(s["dy"], x, stats, s["weight"], x_scales=scales)}
    if op == "pack8":
        codes, scales = kda.kda_pack8(s["x"])
        return {"values": kda.kda_unpack8(codes, scales, dtype=s["io"]), "scales": scales}
    if op == "conv_step":
        return {"y": kda.kda_ssm_conv_step(s["x"], s["w"], s["conv_state"], bias=s["bias"]),
                "conv_state": s["conv_state"]}
    if op == "conv_train":
        y, last = kda.kda_ssm_conv(s["x"], s["w"], s["cu"], bias=s["bias"], conv_state_in=s["conv_state"],
                                   output_conv_state=True)
        return {"y": y, "conv_state": last,
                **kda.kda_ssm_conv_backward(s["x"], s["w"], s["cu"], s["dy"], bias=s["bias"],
                                            conv_state_in=s["conv_state"])}
    ins = (s["u"], s["dt"], s["A"], s["B"], s["C"])
    more = dict(D=s["D"], z=s["z"], dt_bias=s["dt_bias"])
    if op == "step":
        return {"y": kda.kda_ssm_step(*ins, s["state"], **more), "state": s["state"]}
    y, final = kda.kda_ssm_scan(*ins, s["cu"], initial_state=s["state"], **more)
    if op == "scan":
        return {"y": y, "final_state": final}
    return {"y": y, "final_state": final,
            **kda.kda_ssm_backward(*ins, s["cu"], s["dy"], initial_state=s["state"], **more)}


def run(state):
    return _own(state) if own else _PLAIN[state["op"]](state)


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    op, b = case["op"], 2 if case["io"] == "bf16" else 4
    if op in ("norm", "norm_train", "pack8"):
        n, w = case["rows"] * case["width"], case["width"]
        if op == "norm":
            return {"bytes": 2 * b * n + 8 * w, "flops": 8 * n}
        if op == "pack8":  # x in, codes and scales out and in, values out
            return {"bytes": 2 * b * n + 2 * (n + n / 32), "flops": 5 * n}
        kept = 2 * (n + n / 32) if case["saved"] == "e4m3" else 0
        return {"bytes": 4 * b * n + kept + 16 * w, "flops": 22 * n}
    ch = case["ch"]
    if op == "conv_step":
        n = case["batch"] * ch
        return {"bytes": n * b * (1 + 3 + 3 + 1) + 20 * ch, "flops": 14 * n}
    if op == "conv_train":
        lens = [int(v) for v in case["lens"].split(",")]
        n = sum(lens) * ch
        st = len(lens) * ch * 3 * (b + ((b + 4) if case["state"] else 0))
        return {"bytes": n * b * 4 + st + 40 * ch, "flops": 44 * n}
    N, G = case["n"], case["groups"]
    gate = 1 if case["gate"] else 0
    if op == "step":
        n = case["batch"] * ch
        return {"bytes": n * (8 * N + b * (3 + gate)) + 2 * case["batch"] * G * N * b + 4 * ch * (N + 2), "flops": n * (7 * N + 12)}
    lens = [int(v) for v in case["lens"].split(",")]
    T = sum(lens)
    n, rows, st = T * ch, T * G * N * b, 4 * len(lens) * ch * N
    if op == "scan":
        return {"bytes": n * b * (3 + gate) + 2 * rows + st * (2 if case["state"] else 1) + 4 * ch * (N + 2), "flops": n * (7 * N + 12)}
    return {"bytes": n * b * (6 + 2 * gate) + 4 * rows + st * (3 if case["state"] else 1) + 8 * ch * (N + 2), "flops": n * (26 * N + 40)}


# ------------------------------------------------------------------ the definition in 64 bits
def _e4m3(v):
    """fp64 values of magnitude at most 448, rounded to e4m3 (ties to the even code)."""
    step = torch.exp2(torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -6))) - 3)
    return torch.round(v / step) * step


def _exact_pack8(x):
    M, W = x.shape
    v = torch.zeros(M, -(-W // 32) * 32, dtype=torch.float64, device=x.device)
    v[:, :W] = x.double()
    v = v.view(M, -1, 32)
    top = v.abs().amax(2, keepdim=True)
    e = torch.ceil(torch.log2((top / 448).clamp(min=2.0 ** -126)))
    e = torch.where(top > 448 * torch.exp2(e), e + 1, e)
    e = torch.where((top <= 448 * torch.exp2(e - 1)) & (e > -126), e - 1, e)
    back = (_e4m3(v / torch.exp2(e)) * torch.exp2(e)).view(M, -1)[:, :W]
    return back, (e.view(M, -1) + 127).to(torch.uint8)


def _exact_norm(s):
    x = s["x"].double()
    W = x.shape[1]
    mean = x.sum(1, keepdim=True) / W
    var = (x * x).sum(1, keepdim=True) / W - mean * mean
    r = 1 / torch.sqrt(var + EPS)
    y = (x - mean) * r * s["weight"].double() + s["bias"].double()
    if s["op"] == "norm":
        return y
    if s["saved"] == "e4m3":
        x = _exact_pack8(s["x"])[0]
    dy, w, n = s["dy"].double(), s["weight"].double(), (x - mean) * r
    dn = dy * w
    dx = (dn - dn.sum(1, keepdim=True) / W - n * ((dn * n).sum(1, keepdim=True) / W)) * r
    return {"y": y, "dx": dx, "dweight": torch.einsum("mc,mc->c", dy, n), "dbias": torch.einsum("mc->c", dy)}


def _exact_conv_train(s):
    host, x, w = s["cu"][1], s["x"].double(), s["w"].double()
    Ch, N = x.shape[1], len(host) - 1
    y, dx = torch.empty_like(x), torch.empty_like(x)
    dw, db = torch.zeros_like(w), torch.zeros(Ch, dtype=torch.float64, device=x.device)
    last = torch.empty(N, Ch, 3, dtype=torch.float64, device=x.device)
    dst = torch.empty_like(last)
    for i in range(N):
        a, b = int(host[i]), int(host[i + 1])
        old = torch.zeros(3, Ch, dtype=torch.float64, device=x.device) if s["conv_state"] is None else s["conv_state"][i].double().t()
        xs = torch.cat([old, x[a:b]])
        L = b - a
        pre = s["bias"].double() + sum(xs[j:j + L] * w[:, j] for j in range(4))
        y[a:b] = pre / (1 + torch.exp(-pre))
        e = torch.exp(-pre)
        d = s["dy"][a:b].double() * ((1 + e + pre * e) / (1 + e) ** 2)
        dxs = torch.zeros_like(xs)
        for j in range(4):
            dxs[j:j + L] += d * w[:, j]
            dw[:, j] += (d * xs[j:j + L]).sum(0)
        db += d.sum(0)
        dx[a:b], dst[i], last[i] = dxs[3:], dxs[:3].t(), xs[-3:].t()
    out = {"y": y, "dx": dx, "dw": dw, "dbias": db, "conv_state": last}
    if s["conv_state"] is not None:
        out["dconv_state_in"] = dst
    return out


def _exact_scan(s):
    """Token by token, all sequences that are long enough at once."""
    host, dev = s["cu"][1], s["u"].device
    lens = np.diff(host)
    order = np.argsort(-lens, kind="stable")
    begin = torch.from_numpy(np.ascontiguousarray(host[:-1][order]).astype(np.int64)).to(dev)
    live = [int((lens > t).sum()) for t in range(int(lens.max()))]
    u, A, D = s["u"].double(), s["A"].double(), s["D"].double()
    T, Ch = u.shape
    N, G = A.shape[1], s["B"].shape[1]
    x = s["dt"].double() + s["dt_bias"].double()
    delta = torch.logaddexp(x, torch.zeros_like(x))
    B, C = s["B"].double(), s["C"].double()
    rows = lambda v, r: v[r].unsqueeze(2).expand(len(r), G, Ch // G, N).reshape(len(r), Ch, N)  # noqa: E731
    st0 = torch.zeros(len(lens), Ch, N, dtype=torch.float64, device=dev) if s["state"] is None else s["state"].double()
    h = st0[torch.from_numpy(order).to(dev)]
    train = s["op"] == "scan_train"
    hist = torch.empty(T, Ch, N, dtype=torch.float64, device=dev) if train else None
    ybar = torch.empty_like(u)
    for t, k in enumerate(live):
        r = begin[:k] + t
        h[:k] = torch.exp(delta[r].unsqueeze(2) * A) * h[:k] + (delta[r] * u[r]).unsqueeze(2) * rows(B, r)
        ybar[r] = (rows(C, r) * h[:k]).sum(2) + D * u[r]
        if train:
            hist[r] = h[:k]
    final = torch.empty_like(h)
    final[torch.from_numpy(order).to(dev)] = h
    z = None if s["z"] is None else s["z"].double()
    y = ybar if z is None else ybar * z / (1 + torch.exp(-z))
    if not train:
        return {"y": y, "final_state": final}
    dy = s["dy"].double()
    out = {"y": y, "final_state": final}
    g = dy
    if z is not None:
        e = torch.exp(-z)
        out["dz"] = dy * ybar * ((1 + e + z * e) / (1 + e) ** 2)
        g = dy * z / (1 + e)
    dB, dC = torch.empty(T, G, N, dtype=torch.float64, device=dev), torch.empty(T, G, N, dtype=torch.float64, device=dev)
    du, dx, dA = torch.empty_like(u), torch.empty_like(u), torch.zeros_like(A)
    q = torch.zeros_like(h)  # a_{t+1} times the gradient of h_{t+1}
    start = st0[torch.from_numpy(order).to(dev)]
    for t in range(len(live) - 1, -1, -1):
        k = live[t]
        r = begin[:k] + t
        before = hist[r - 1] if t else start[:k]
        a = torch.exp(delta[r].unsqueeze(2) * A)
        lam = q[:k] + g[r].unsqueeze(2) * rows(C, r)
        dC[r] = (g[r].unsqueeze(2) * hist[r]).view(k, G, Ch // G, N).sum(2)
        dB[r] = (lam * (delta[r] * u[r]).unsqueeze(2)).view(k, G, Ch // G, N).sum(2)
        through = (lam * rows(B, r)).sum(2)
        da = lam * before * a
        dA += (da * delta[r].unsqueeze(2)).sum(0)
        du[r] = through * delta[r] + g[r] * D
        dx[r] = (through * u[r] + (da * A).sum(2)) / (1 + torch.exp(-x[r]))
        q[:k] = a * lam
    out |= {"dA": dA, "dB": dB, "dC": dC, "du": du, "ddt": dx, "ddt_bias": dx.sum(0), "dD": (g * u).sum(0)}
    if s["state"] is not None:
        dinit = torch.empty_like(q)
        dinit[torch.from_numpy(order).to(dev)] = q
        out["dinitial_state"] = dinit
    return out


def _exact_step(s):
    u, A = s["u"].double(), s["A"].double()
    x = s["dt"].double() + s["dt_bias"].double()
    delta = torch.logaddexp(x, torch.zeros_like(x))
    M, Ch = u.shape
    G, N = s["B"].shape[1:]
    wide = lambda v: v.double().unsqueeze(2).expand(M, G, Ch // G, N).reshape(M, Ch, N)  # noqa: E731
    h = torch.exp(delta.unsqueeze(2) * A) * s["state"].double() + (delta * u).unsqueeze(2) * wide(s["B"])
    y = torch.einsum("mcn,mcn->mc", h, wide(s["C"])) + s["D"].double() * u
    if s["z"] is not None:
        z = s["z"].double()
        y = y * z / (1 + torch.exp(-z))
    return {"y": y, "state": h}


def exact(case, seed):
    s, op = prepare(case, seed), case["op"]
    if op in ("norm", "norm_train"):
        return _exact_norm(s)
    if op == "pack8":
        values, scales = _exact_pack8(s["x"])
        return {"values": values, "scales": scales}
    if op == "conv_step":
        win = torch.cat([s["conv_state"], s["x"].unsqueeze(2)], 2).double()
        pre = torch.einsum("mcj,cj->mc", win, s["w"].double()) + s["bias"].double()
        return {"y": pre / (1 + torch.exp(-pre)), "conv_state": win[:, :, 1:]}
    if op == "conv_train":
        return _exact_conv_train(s)
    return _exact_step(s) if op == "step" else _exact_scan(s)
