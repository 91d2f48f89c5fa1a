"""Plain 64-bit forms of the operators of a decode step over few tokens (4-bit weights, the mixture of experts, the
verification of drafts), on the CPU, and the error bounds that their tests use.

Bounds: a value stored in a type is off by at most half a step, u = eps / 2 relative (bf16 2^-8, fp32 2^-24).  A product
with 4-bit weights adds products that are exact in fp32 (16-bit operands of at most 8 + 4 bits): 32 of them in two
matrix instructions, whose sums may drop what lies below 2^-23 of their largest term, then one multiply-add per group of
32 and one per 256; so |error| <= (K / 32 + 16) 2^-23 sum |x w|, counting every one at a full step of the whole sum.
"""
from __future__ import annotations

import numpy as np
import torch

from block_testlib import U, f64, gen, randn, within  # noqa: F401

E2M1 = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64)
FORMATS = [("e2m1", 32, None), ("int4", 32, torch.bfloat16), ("int4", 64, torch.float32), ("int4", 128, torch.bfloat16)]


def unpack_ref(codes, scales):
    """The weights that codes and scales stand for, fp64."""
    codes = codes.cpu()
    c = torch.stack([codes & 15, codes >> 4], -1).view(*codes.shape[:-1], -1).long()
    if scales.dtype == torch.uint8:
        v = torch.cat([E2M1, -E2M1])[c]
        s = torch.exp2(scales.cpu().double() - 127)
    else:
        v, s = (c - 8).double(), f64(scales)
    return v * s.repeat_interleave(c.shape[-1] // s.shape[-1], -1)


def pack_ref(w, fmt, group, scale_dtype):
    """Codes (one per weight) and scales of fp64 weights [rows, K]."""
    g = f64(w).view(w.shape[0], -1, group)
    top = g.abs().amax(2, keepdim=True)
    if fmt == "e2m1":
        e = torch.full_like(top, -126.0)
        for k in range(-126, 127):  # the smallest power of two with top <= 6 * 2^k
            e = torch.where(top > 6 * 2.0 ** (k - 1), torch.full_like(e, float(max(k, -126))), e)
        v = g / torch.exp2(e)
        a = v.abs()
        # nearest value, ties to the even code
        d = (a.unsqueeze(-1) - E2M1).abs()
        near = d.amin(-1, keepdim=True)
        cand = (d == near)
        idx = torch.arange(8)
        even = torch.where(cand & (idx % 2 == 0), idx, 99).amin(-1)
        code = torch.where(even < 99, even, torch.where(cand, idx, 99).amin(-1))
        code = code + 8 * (torch.signbit(v)).long()
        return code.view(w.shape), (e[..., 0] + 127).to(torch.uint8)
    s = (top / 7).float().to(scale_dtype)
    sd = s.double()
    code = torch.where(sd > 0, torch.round((g.float() / s.float()).double()).clamp(-8, 7), torch.zeros_like(g)) + 8
    return code.long().view(w.shape), s[..., 0]


def random_weight(g, *shape, fmt, group, scale_dtype=None, std=None):
    """Random codes and scales for weights [..., K] of about K^-1/2."""
    *lead, K = shape
    std = K ** -0.5 if std is None else std
    codes = torch.randint(0, 256, (*lead, K // 2), generator=g, dtype=torch.uint8)
    if fmt == "e2m1":
        e = torch.randn(*lead, K // group, generator=g) + float(np.log2(std / 3))
        return codes, (torch.round(e).clamp(-120, 120) + 127).to(torch.uint8)
    return codes, (torch.exp(0.3 * torch.randn(*lead, K // group, generator=g)) * (std / 5)).to(scale_dtype)


def gemm4_ref(x, w, epilogue):
    """(result, bound before the rounding to the output's type)."""
    x, w = f64(x), f64(w)
    y, mass = x @ w.t(), x.abs() @ w.abs().t()
    err = (x.shape[1] / 32 + 16) * 2.0 ** -23 * mass
    if epilogue == "none":
        return y, err
    sg, top = torch.sigmoid(y), 5.0 if epilogue == "decay" else 1.0
    # |sigmoid'| <= 1/4; the exponential, the sum and the quotient are off by a few units of 2^-24
    return (-5 * sg if epilogue == "decay" else sg), top * (err / 4 + 8 * 2.0 ** -24 * sg)


def moe_ref(x, router, w_in, w_out, top, bias, score, scale):
    """y, ids, weights and the bound of y, from fp64 weights w_in [E, 2F, D] and w_out [E, D, F]."""
    x, logits = f64(x), f64(x) @ f64(router).t()
    M, E = logits.shape
    s = torch.sigmoid(logits) if score == "sigmoid" else logits
    key = s if bias is None else s + f64(bias)
    key = torch.where(torch.isnan(key), torch.full_like(key, -torch.inf), key)
    ids = torch.from_numpy(np.lexsort((np.broadcast_to(np.arange(E), (M, E)), -key.numpy()), axis=1)[:, :top].copy())
    w = s.gather(1, ids)
    if score == "softmax":
        w = torch.exp(w - w[:, :1])
    w = scale * w / w.sum(1, keepdim=True)
    y, bound = torch.zeros_like(x), torch.zeros_like(x)
    D, F = w_out.shape[1], w_out.shape[2]
    for t in range(M):
        for j in range(top):
            e = int(ids[t, j])
            gu = w_in[e] @ x[t]
            dgu = (D / 32 + 16) * 2.0 ** -23 * (w_in[e].abs() @ x[t].abs())
            g, u, dg, du = gu[:F], gu[F:], dgu[:F], dgu[F:]
            sg = torch.sigmoid(g)
            h = g * sg * u
            # |silu'| <= 1.1; the activation's own operations a few units of 2^-24
            dh = 1.1 * dg * (u.abs() + du) + (g * sg).abs() * du + 12 * 2.0 ** -24 * h.abs()
            # fp32 hidden values enter the product in terms of 22 bits at least (and 2^-36 of a run's largest)
            dh = dh + 2.0 ** -21 * h.abs() + 2.0 ** -36 * h.abs().max()
            p = w_out[e] @ h
            dp = w_out[e].abs() @ dh + (F / 32 + 16) * 2.0 ** -23 * (w_out[e].abs() @ (h.abs() + dh))
            y[t] += w[t, j] * p
            bound[t] += w[t, j].abs() * (dp + 8 * 2.0 ** -24 * p.abs())
    return y, ids, w, bound + top * 2.0 ** -23 * bound.sign() * y.abs()


def verify_ref(target, draft, tokens, u, cu):
    T, V = target.shape
    pos = lambda r: torch.where(f64(r) > 0, f64(r), torch.zeros(V, dtype=torch.float64))  # noqa: E731
    out, accepted = np.full(T, -1, np.int64), np.zeros(len(cu) - 1, np.int32)
    for n in range(len(cu) - 1):
        a, b = int(cu[n]), int(cu[n + 1])
        if a == b:
            continue
        i = a
        while i < b - 1:
            d = int(tokens[i])
            if not 0 <= d < V:
                break
            q = 1.0 if draft is None else float(draft[i, d])
            if not float(u[i]) * q < float(target[i, d]):
                break
            out[i] = d
            i += 1
        rest = pos(target[i])
        if i < b - 1:
            left = rest.clone()
            if draft is not None:
                left = (rest - pos(draft[i])).clamp(min=0)
            elif 0 <= int(tokens[i]) < V:
                left[int(tokens[i])] = 0
            rest = left if left.sum() > 0 else rest
        cum = torch.cumsum(rest, 0)
        if cum[-1] > 0:
            over = torch.nonzero(cum > float(u[b - 1]) * cum[-1])
            out[i] = int(over[0]) if len(over) else int(torch.nonzero(rest > 0)[-1])
        accepted[n] = i - a
    return out, accepted
