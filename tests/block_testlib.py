"""Plain 64-bit forms of the operators around the layer (layer norm, 8-bit activations, the short convolution and the
selective state space scan), on the CPU, and the error bounds that their tests use.

Rounding bounds: a value stored in a type is off by at most half a step, u = eps / 2 relative (bf16 2^-8, fp32 2^-24,
e4m3 2^-4).  Arithmetic is fp32 throughout, so every bound is c * 2^-24 times the magnitude that the sums run over, plus
one rounding to the output's type.
"""
from __future__ import annotations

import numpy as np
import torch

U32 = 2.0 ** -24
U = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}


def f64(t):
    return None if t is None else t.detach().to("cpu", torch.float64)


def gen(seed):
    g = torch.Generator()
    g.manual_seed(seed)
    return g


def randn(g, *shape, std=1.0, mean=0.0, dtype=torch.float32):
    return (torch.randn(*shape, generator=g) * std + mean).to(dtype)


def within(got, ref, bound, what=""):
    """|got - ref| <= bound elementwise (bound broadcasts); NaN where and only where the reference has NaN."""
    got, ref = f64(got), f64(ref)
    assert got.shape == ref.shape, f"{what}: shape {tuple(got.shape)} vs {tuple(ref.shape)}"
    assert torch.equal(torch.isnan(got), torch.isnan(ref)), f"{what}: NaN in other places"
    over = ((got - ref).abs() - bound).nan_to_num(nan=-1.0)
    if over.numel() and over.max() > 0:
        i = int(over.argmax())
        raise AssertionError(f"{what}: off by {(got - ref).abs().flatten()[i]:.3e} at {i}: got "
                             f"{got.flatten()[i]:.9e}, want {ref.flatten()[i]:.9e}")


# ------------------------------------------------------------------ layer norm
def norm_ref(x, w, b, eps, dy=None, x_bwd=None):
    """y, mean, rstd and, with dy, dx, dw, db; x_bwd: the x that the backward pass reads (default x)."""
    x = f64(x)
    w = torch.ones(x.shape[1], dtype=torch.float64) if w is None else f64(w)
    b = torch.zeros(x.shape[1], dtype=torch.float64) if b is None else f64(b)
    mean = x.mean(1, keepdim=True)
    rstd = 1 / torch.sqrt(((x - mean) ** 2).mean(1, keepdim=True) + eps)
    out = {"y": (x - mean) * rstd * w + b, "mean": mean[:, 0], "rstd": rstd[:, 0]}
    if dy is not None:
        dy = f64(dy)
        xh = ((x if x_bwd is None else f64(x_bwd)) - mean) * rstd
        p = dy * w
        out["dx"] = rstd * (p - p.mean(1, keepdim=True) - xh * (p * xh).mean(1, keepdim=True))
        out["dweight"], out["dbias"] = (dy * xh).sum(0), dy.sum(0)
    return out


# ------------------------------------------------------------------ 8 bits
def pack8_ref(x):
    """(values, scale bytes) by the definition: per 32 channels the smallest e >= -126 with max|x| <= 448 2^e."""
    x = f64(x).numpy()
    M, C = x.shape
    nb = -(-C // 32)
    v = np.zeros((M, nb * 32))
    v[:, :C] = x
    v = v.reshape(M, nb, 32)
    finite = np.isfinite(v)
    top = np.abs(np.where(finite, v, 0)).max(2)
    e = np.full(top.shape, -126, np.int64)
    with np.errstate(divide="ignore"):
        guess = np.where(top > 0, np.floor(np.log2(np.maximum(top, 1e-300))) - 9, -200).astype(np.int64)
    for step in range(4):  # the smallest exponent that holds the maximum, searched upwards
        cand = guess + step
        fits = top <= 448 * np.exp2(cand.astype(np.float64))
        e = np.where((e == -126) & fits & (cand >= -126), cand, e)
        guess = np.where(fits, -10000, guess)
    s = np.exp2(e.astype(np.float64))[:, :, None]
    q = np.where(finite, v, 0) / s
    step = np.exp2(np.floor(np.log2(np.maximum(np.abs(q), 2.0 ** -6))) - 3)
    back = np.where(finite, np.rint(q / step) * step * s, np.nan)
    return torch.from_numpy(back.reshape(M, -1)[:, :C].copy()), torch.from_numpy((e + 127).astype(np.uint8))


# ------------------------------------------------------------------ the short convolution
def conv_ref(x, w, bias, lens, silu, state=None, dy=None):
    """y, the conv states that the sequences leave, and, with dy, dx, dw, dbias and dstate."""
    x, w = f64(x), f64(w)
    C = x.shape[1]
    b = torch.zeros(C, dtype=torch.float64) if bias is None else f64(bias)
    y, last = torch.empty_like(x), torch.zeros(len(lens), C, 3, dtype=torch.float64)
    out = {"y": y, "state": last}
    if dy is not None:
        dy = f64(dy)
        out |= {"dx": torch.empty_like(x), "dw": torch.zeros_like(w), "dbias": torch.zeros(C, dtype=torch.float64),
                "dstate": torch.zeros_like(last)}
    t0 = 0
    for i, L in enumerate(lens):
        old = torch.zeros(3, C, dtype=torch.float64) if state is None else f64(state)[i].t()
        xs = torch.cat([old, x[t0:t0 + L]])
        last[i] = xs[L:L + 3].t()
        pre = b + sum(xs[j:j + L] * w[:, j] for j in range(4))
        sg = torch.sigmoid(pre)
        y[t0:t0 + L] = pre * sg if silu else pre
        if dy is not None:
            d = dy[t0:t0 + L] * (sg * (1 + pre * (1 - sg)) if silu else 1.0)
            dxs = torch.zeros_like(xs)
            for j in range(4):
                dxs[j:j + L] += d * w[:, j]
                out["dw"][:, j] += (d * xs[j:j + L]).sum(0)
            out["dbias"] += d.sum(0)
            out["dstate"][i], out["dx"][t0:t0 + L] = dxs[:3].t(), dxs[3:]
        t0 += L
    return out


# ------------------------------------------------------------------ the selective scan
def ssm_ref(u, dt, A, B, C, lens, D=None, z=None, dt_bias=None, softplus=True, init=None):
    """(y, final_state) token by token; differentiable by autograd when the inputs are 64-bit leaves."""
    f = lambda t: None if t is None else t.to("cpu", torch.float64)  # noqa: E731
    u, dt, A, B, C, D, z, dt_bias, init = map(f, (u, dt, A, B, C, D, z, dt_bias, init))
    T, Ch = u.shape
    N, G = A.shape[1], B.shape[1]
    x = dt if dt_bias is None else dt + dt_bias
    delta = torch.logaddexp(x, torch.zeros_like(x)) if softplus else x
    wide = lambda r: r.unsqueeze(1).expand(G, Ch // G, N).reshape(Ch, N)  # noqa: E731
    ys, finals, t = [], [], 0
    for i, L in enumerate(lens):
        h = torch.zeros(Ch, N, dtype=torch.float64) if init is None else init[i]
        for t in range(t, t + L):
            h = torch.exp(delta[t].unsqueeze(1) * A) * h + (delta[t] * u[t]).unsqueeze(1) * wide(B[t])
            y = (wide(C[t]) * h).sum(1)
            ys.append(y if D is None else y + D * u[t])
        t = t + 1 if L else t
        finals.append(h)
    y = torch.stack(ys) if ys else torch.zeros(0, Ch, dtype=torch.float64)
    if z is not None:
        y = y * z * torch.sigmoid(z)
    return y, torch.stack(finals) if finals else torch.zeros(0, Ch, N, dtype=torch.float64)


def ssm_inputs(seed, T, Ch, N, G, io, n_seq=1, gate=True, skip=True, bias=True, state=True, slow=False):
    """Inputs of the scan as trained ones spread; slow: step sizes near 1e-3, so a state remembers a thousand tokens."""
    g = gen(seed)
    lo, hi = (1e-3, 2e-3) if slow else (1e-3, 1e-1)
    step = torch.exp(torch.rand(Ch, generator=g) * float(np.log(hi / lo)) + float(np.log(lo)))
    return dict(u=randn(g, T, Ch, dtype=io), dt=randn(g, T, Ch, std=0.5, dtype=io),
                A=-torch.arange(1, N + 1).float() * torch.exp(randn(g, Ch, N, std=0.1)),
                B=randn(g, T, G, N, dtype=io), C=randn(g, T, G, N, dtype=io),
                D=randn(g, Ch) if skip else None, z=randn(g, T, Ch, dtype=io) if gate else None,
                dt_bias=(step + torch.log(-torch.expm1(-step))) if bias else None,
                init=randn(g, n_seq, Ch, N) if state else None)
