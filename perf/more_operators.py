"""The operators of a decode step over few tokens, as one measured set: projections with 4-bit weights, a
mixture-of-experts layer, and the verification of drafted tokens.

Each case is one pass through one operator.  ``run`` computes it in plain torch operations (fp32, and fp64 where a
choice hangs on the last digits; rounded once at the end) or, with ``own`` set, through the package's entry points;
``exact`` computes it in 64 bits.
"""
import math

import numpy as np
import torch

own = False

_DT = {"bf16": torch.bfloat16, "fp32": torch.float32}
# the sixteen e2m1 values by code: sign, two bits of exponent, one of mantissa
_E2M1 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0]


# ------------------------------------------------------------------ cases
def listed():
    return [
        # one token through the query projection, 7,168 -> 12,288, weights as they are stored in 4 bits
        dict(name="gemm4_token", op="gemm4", rows=1, n=12288, k=7168, fmt="e2m1", group=32, epi="none", out="bf16"),
        # eight sequences that verify three drafted tokens each
        dict(name="gemm4_verify_8x4", op="gemm4", rows=32, n=12288, k=7168, fmt="e2m1", group=32, epi="none", out="bf16"),
        # the decode step of 256 sequences, out projection
        dict(name="gemm4_decode_256", op="gemm4", rows=256, n=7168, k=12288, fmt="e2m1", group=32, epi="none", out="bf16"),
        # a vocabulary's worth of rows for 16 tokens, integer codes with one scale for 128 weights
        dict(name="gemm4_vocabulary", op="gemm4", rows=16, n=160000, k=7168, fmt="int4", group=128, epi="none", out="fp32"),
        # the log-decay of five tokens, odd sizes
        dict(name="gemm4_decay_odd", op="gemm4", rows=5, n=1001, k=1056, fmt="int4", group=32, epi="decay", out="fp32"),
        # one token through 16 of 896 experts
        dict(name="moe_token", op="moe", rows=1, experts=896, top=16, d=3584, f=2048, fmt="e2m1", group=32, score="sigmoid",
             out="bf16"),
        # eight sequences of four tokens through 8 of 256 experts
        dict(name="moe_verify_8x4", op="moe", rows=32, experts=256, top=8, d=7168, f=2048, fmt="e2m1", group=32,
             score="sigmoid", out="bf16"),
        # experts that were left in bf16, softmax scores
        dict(name="moe_bf16", op="moe", rows=4, experts=64, top=6, d=2048, f=1408, fmt="bf16", group=0, score="softmax",
             out="fp32"),
        # odd sizes, integer codes
        dict(name="moe_odd", op="moe", rows=7, experts=33, top=3, d=1056, f=352, fmt="int4", group=32, score="sigmoid",
             out="bf16"),
        # 256 sequences of four tokens: three drafts each
        dict(name="verify_256x4", op="verify", lens=",".join(["4"] * 256), vocab=160000, probs="fp32", draft=True),
        # a single sequence with seven drafts
        dict(name="verify_1x8", op="verify", lens="8", vocab=160000, probs="fp32", draft=True),
        # ragged batch, an odd vocabulary, a drafter that proposes its best token only
        dict(name="verify_ragged_greedy", op="verify", lens="5,1,2,8,3,1,6,4,2,7,1", vocab=32003, probs="bf16", draft=False),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _format(rng, k, kinds):
    """A format and a group that divides k (a multiple of 32)."""
    fmt = rng.choice(kinds)
    if fmt != "int4":
        return fmt, 32 if fmt == "e2m1" else 0
    return fmt, rng.choice([g for g in (32, 64, 128) if k % g == 0])


def draw(rng):
    op = rng.choice(["gemm4", "gemm4", "moe", "moe", "verify"])
    out = rng.choice(["bf16", "bf16", "fp32"])
    if op == "gemm4":
        k = 32 * _log_int(rng, 2, 448)
        n = _log_int(rng, 16, min(160000, (1 << 27) // k))
        rows = _log_int(rng, 1, 256)
        fmt, group = _format(rng, k, ["e2m1", "int4"])
        return dict(op=op, rows=rows, n=n, k=k, fmt=fmt, group=group, epi=rng.choice(["none", "none", "decay", "sigmoid"]),
                    out=out)
    if op == "moe":
        unit = rng.choice([32, 64, 128])
        d, f = unit * _log_int(rng, 4, 7168 // unit), unit * _log_int(rng, 2, 2048 // unit)
        fmt, group = _format(rng, unit, ["e2m1", "e2m1", "int4", "bf16"])
        most = (1 << 33) // (d * f * (4 if fmt == "bf16" else 1))  # all experts: 13 GB at most
        experts = _log_int(rng, 2, max(2, min(896, most)))
        top = rng.randint(1, min(16, experts))
        return dict(op=op, rows=_log_int(rng, 1, max(1, min(64, 512 // top))), experts=experts, top=top, d=d, f=f, fmt=fmt,
                    group=group, score=rng.choice(["sigmoid", "softmax"]), out=out)
    vocab = _log_int(rng, 100, 160000)
    n = _log_int(rng, 1, 256)
    lens = [rng.randint(1, 8) for _ in range(n)]
    while sum(lens) * vocab > 1024 * 160000:
        lens.pop()
    if rng.random() < 0.3:
        lens[rng.randrange(len(lens))] = 0  # a slot of the batch without a sequence
    return dict(op=op, lens=",".join(map(str, lens)), vocab=vocab, probs=rng.choice(["fp32", "fp32", "bf16"]),
                draft=rng.random() < 0.7)


# ------------------------------------------------------------------ inputs
class _Maker:
    def __init__(self, seed):
        self.g = torch.Generator(device="cuda")
        self.g.manual_seed(int(seed))

    def normal(self, *shape, std=1.0, mean=0.0, dtype=torch.float32):
        return (torch.randn(*shape, generator=self.g, device="cuda") * std + mean).to(dtype)

    def uniform(self, *shape, lo=0.0, hi=1.0, dtype=torch.float32):
        return (torch.rand(*shape, generator=self.g, device="cuda") * (hi - lo) + lo).to(dtype)

    def codes(self, *shape, fmt):
        """Two codes per byte, the even one low, distributed as the codes of normal weights are."""
        z = torch.special.ndtri((torch.arange(256, device="cuda", dtype=torch.float64) + 0.5) / 256)
        if fmt == "int4":
            code = torch.round(z * 2.6).clamp(-7, 7).long() + 8
        else:
            table = torch.tensor(_E2M1, device="cuda", dtype=torch.float64)
            code = (z.mul(1.9).clamp(-6, 6).unsqueeze(1) - table).abs().argmin(1)
        pair = (code.unsqueeze(0) | (code.unsqueeze(1) << 4)).to(torch.uint8).view(-1)  # by two random bytes
        out = torch.empty(shape, dtype=torch.uint8, device="cuda")
        flat, step = out.view(-1), 1 << 28
        for i in range(0, flat.numel(), step):
            part = flat[i:i + step]
            part.copy_(pair[torch.randint(0, 65536, part.shape, generator=self.g, device="cuda", dtype=torch.int32)])
        return out

    def scales(self, *shape, fmt, std):
        """Scales that give weights of about this standard deviation, a factor of a few apart."""
        if fmt == "e2m1":
            e = self.normal(*shape, std=0.6, mean=math.log2(std / 1.9))
            return (torch.round(e).clamp(-60, 60) + 127).to(torch.uint8)
        return torch.exp(self.normal(*shape, std=0.25, mean=math.log(std / 2.6))).to(torch.bfloat16)

    def weight(self, *shape, fmt, group, std):
        if fmt == "bf16":
            out = torch.empty(shape, dtype=torch.bfloat16, device="cuda")
            for part in out.view(shape[0], -1).split(max(1, (1 << 27) // (out.numel() // shape[0]))):
                part.copy_(self.normal(*part.shape, std=std))
            return out
        *lead, k = shape
        return self.codes(*lead, k // 2, fmt=fmt), self.scales(*lead, k // group, fmt=fmt, std=std)


def prepare(case, seed):
    m, op = _Maker(seed), case["op"]
    s = {"op": op}
    if op == "gemm4":
        K = case["k"]
        s["x"] = m.normal(case["rows"], K, dtype=torch.bfloat16)
        s["w"] = m.weight(case["n"], K, fmt=case["fmt"], group=case["group"], std=K ** -0.5)
        s["epi"], s["out"] = case["epi"], _DT[case["out"]]
        return s
    if op == "moe":
        E, D, F = case["experts"], case["d"], case["f"]
        s["x"] = m.normal(case["rows"], D, dtype=torch.bfloat16)
        s["router"] = m.normal(E, D, std=D ** -0.5, dtype=torch.bfloat16)
        s["bias"] = m.normal(E, std=0.02) if case["score"] == "sigmoid" else None
        s["w_in"] = m.weight(E, 2 * F, D, fmt=case["fmt"], group=case["group"], std=D ** -0.5)
        s["w_out"] = m.weight(E, D, F, fmt=case["fmt"], group=case["group"], std=F ** -0.5)
        s["top"], s["score"], s["out"] = case["top"], case["score"], _DT[case["out"]]
        return s
    lens = [int(v) for v in case["lens"].split(",")]
    host = np.zeros(len(lens) + 1, np.int32)
    host[1:] = np.cumsum(lens)
    s["cu"] = (torch.from_numpy(host).cuda(), host)
    T, V = int(host[-1]), case["vocab"]
    # a peaked distribution, and a drafter that agrees with it for the most part
    logits = m.normal(T, V, std=2.5)
    near = logits + m.normal(T, V, std=0.7)
    s["target"] = torch.softmax(logits, 1).to(_DT[case["probs"]])
    if case["draft"]:
        near = torch.softmax(near, 1)
        s["draft"] = near.to(_DT[case["probs"]])
        s["tokens"] = (near / -torch.log(m.uniform(T, V).clamp(min=1e-30))).argmax(1).int()
    else:
        s["draft"], s["tokens"] = None, near.argmax(1).int()
        hot = torch.zeros(T, V, device="cuda").scatter_(1, s["tokens"].long().unsqueeze(1), 1.0)
        s["target"] = (0.5 * s["target"].float() + 0.5 * hot).to(_DT[case["probs"]])
    s["u"] = m.uniform(T)
    return s


# ------------------------------------------------------------------ the plain forms
def _plain_weight(w):
    """fp32 values of a bf16 weight or of 4-bit codes and their scales."""
    if isinstance(w, torch.Tensor):
        return w.float()
    codes, scales = w
    if scales.dtype == torch.uint8:
        table = torch.tensor(_E2M1, device=codes.device)
        factor = torch.exp2(scales.float() - 127)
    else:
        table = torch.arange(-8, 8, device=codes.device, dtype=torch.float32)
        factor = scales.float()
    v = torch.stack([table[(codes & 15).int()], table[(codes >> 4).int()]], -1)
    v = v.view(*scales.shape, -1) * factor.unsqueeze(-1)
    return v.view(*codes.shape[:-1], -1)


def _plain_gemm4(s):
    y = s["x"].float() @ _plain_weight(s["w"]).t()
    if s["epi"] == "decay":
        y = -5 * torch.sigmoid(y)
    elif s["epi"] == "sigmoid":
        y = torch.sigmoid(y)
    return y.to(s["out"])


def _plain_route(s):
    """Experts and weights of every token, best first; a tie goes to the lower expert."""
    logits = s["x"].double() @ s["router"].double().t()
    score = torch.sigmoid(logits) if s["score"] == "sigmoid" else torch.softmax(logits, 1)
    key = score if s["bias"] is None else score + s["bias"].double()
    ids = torch.sort(key, dim=1, descending=True, stable=True).indices[:, :s["top"]]
    w = score.gather(1, ids)
    return ids, (w / w.sum(1, keepdim=True)).float()


def _plain_moe(s):
    ids, w = _plain_route(s)
    pick = lambda p, e: p[e] if isinstance(p, torch.Tensor) else tuple(t[e] for t in p)  # noqa: E731
    x = s["x"].float()
    y = torch.zeros_like(x)
    for t in range(x.shape[0]):
        for j in range(s["top"]):
            e = ids[t, j:j + 1]
            gate, up = (_plain_weight(pick(s["w_in"], e))[0] @ x[t]).chunk(2)
            y[t] += w[t, j] * (_plain_weight(pick(s["w_out"], e))[0] @ (gate * torch.sigmoid(gate) * up))
    return {"y": y.to(s["out"]), "ids": ids.int(), "weights": w}


def _plain_verify(s):
    cu = s["cu"][0].long()
    p, tokens, u = s["target"], s["tokens"].long(), s["u"].double()
    T, V = p.shape
    rows = torch.arange(T, device=p.device)
    seq = torch.searchsorted(cu, rows, right=True) - 1
    last = cu[seq + 1] - 1
    pd = p.gather(1, tokens.unsqueeze(1))[:, 0].double()
    qd = torch.ones_like(pd) if s["draft"] is None else s["draft"].gather(1, tokens.unsqueeze(1))[:, 0].double()
    stop = (u * qd >= pd) | (rows == last)
    # the first row of each sequence that does not take its draft
    N = cu.shape[0] - 1
    at = torch.full((N,), T, device=p.device).scatter_reduce_(0, seq, torch.where(stop, rows, T), "amin")
    live = cu[1:] > cu[:-1]
    accepted = torch.where(live, at - cu[:-1], 0)
    at = at.clamp(max=T - 1)
    end = (cu[1:] - 1).clamp(min=0)
    full = (at == end).unsqueeze(1)
    own_row = p[at].double()
    if s["draft"] is None:
        rest = own_row.scatter(1, tokens[at].unsqueeze(1), 0.0)
    else:
        rest = (own_row - s["draft"][at].double()).clamp(min=0)
    rest = torch.where(full, own_row, rest)
    cum = rest.cumsum(1)
    drawn = (cum > u[end].unsqueeze(1) * cum[:, -1:]).int().argmax(1)
    out = torch.where(rows < at[seq], tokens, torch.where(rows == at[seq], drawn[seq], -1))
    return {"tokens": out.int(), "accepted": accepted.int()}


_PLAIN = {"gemm4": _plain_gemm4, "moe": _plain_moe, "verify": _plain_verify}


# ------------------------------------------------------------------ the package's operators
def _own(s):
    import kimi_delta_attention_16_gb300 as kda
    if s["op"] == "gemm4":
        return kda.kda_gemm4(s["x"], *s["w"], epilogue=s["epi"], out_dtype=s["out"])
    if s["op"] == "moe":
        y, ids, w = kda.kda_moe(s["x"], s["router"], s["w_in"], s["w_out"], s["top"], bias=s["bias"], score=s["score"],
                                out_dtype=s["out"], return_routing=True)
        return {"y": y, "ids": ids, "weights": w}
    tokens, accepted = kda.kda_verify(s["target"], s["tokens"], s["u"], s["cu"], draft=s["draft"])
    return {"tokens": tokens, "accepted": accepted}


def run(state):
    return _own(state) if own else _PLAIN[state["op"]](state)


# ------------------------------------------------------------------ what a pass cannot do without
def _weight_bytes(case):
    """Bytes of one weight with its share of the scales."""
    return {"bf16": 2.0, "e2m1": 0.5 + 1 / 32}.get(case["fmt"]) or 0.5 + 2 / case["group"]


def work(case):
    op = case["op"]
    if op == "gemm4":
        M, N, K = case["rows"], case["n"], case["k"]
        return {"bytes": N * K * _weight_bytes(case) + 2 * M * K + M * N * (2 if case["out"] == "bf16" else 4),
                "flops": 2 * M * N * K}
    if op == "moe":
        M, E, k, D, F = (case[v] for v in ("rows", "experts", "top", "d", "f"))
        used = E * (1 - (1 - k / E) ** M)  # experts that some token takes, for choices at random
        return {"bytes": used * 3 * D * F * _weight_bytes(case) + 2 * E * D + M * D * (4 if case["out"] == "bf16" else 6),
                "flops": 2 * M * (E * D + 3 * k * D * F)}
    lens = [int(v) for v in case["lens"].split(",")]
    n, b = sum(v > 0 for v in lens), 2 if case["probs"] == "bf16" else 4
    # each sequence reads the one row that it draws from, of both distributions where it can be a rejected one
    both = sum(v > 1 for v in lens) if case["draft"] else 0
    return {"bytes": (n + both) * case["vocab"] * b + sum(lens) * (12 + 2 * b), "flops": 3 * (n + both) * case["vocab"]}


# ------------------------------------------------------------------ the definition in 64 bits
def _exact_weight(w):
    if isinstance(w, torch.Tensor):
        return w.double()
    codes, scales = w
    K = codes.shape[1] * 2
    v = torch.empty(codes.shape[0], K, dtype=torch.float64, device=codes.device)
    for half in (0, 1):
        c = ((codes >> (4 * half)) & 15).double()
        if scales.dtype == torch.uint8:
            sign, c = torch.where(c >= 8, -1.0, 1.0), c % 8
            e = torch.floor(c / 2)
            mant = c - 2 * e
            c = sign * torch.where(e == 0, mant / 2, (1 + mant / 2) * torch.exp2(e - 1))
        else:
            c = c - 8
        v[:, half::2] = c
    f = torch.exp2(scales.double() - 127) if scales.dtype == torch.uint8 else scales.double()
    return v * f.repeat_interleave(K // f.shape[1], 1)


def _exact_gemm4(s):
    codes, scales = s["w"]
    x, parts = s["x"].double(), []
    for i in range(0, codes.shape[0], 16384):
        parts.append(torch.einsum("mk,nk->mn", x, _exact_weight((codes[i:i + 16384], scales[i:i + 16384]))))
    y = torch.cat(parts, 1)
    if s["epi"] == "none":
        return y
    y = 1 / (1 + torch.exp(-y))
    return -5 * y if s["epi"] == "decay" else y


def _exact_moe(s):
    x = s["x"].double()
    M, k = x.shape[0], s["top"]
    logits = torch.einsum("md,ed->me", x, s["router"].double())
    if s["score"] == "sigmoid":
        score = 1 / (1 + torch.exp(-logits))
    else:
        score = torch.exp(logits - logits.amax(1, keepdim=True))
        score = score / score.sum(1, keepdim=True)
    key = (score if s["bias"] is None else score + s["bias"].double()).cpu().numpy()
    score = score.cpu().numpy()
    ids = np.lexsort((np.broadcast_to(np.arange(key.shape[1]), key.shape), -key), axis=1)[:, :k]
    w = np.take_along_axis(score, ids, 1)
    w = w / w.sum(1, keepdims=True)
    y = torch.zeros_like(x)
    for e in np.unique(ids):
        t, j = np.nonzero(ids == e)
        one = lambda p: p[e] if isinstance(p, torch.Tensor) else (p[0][e], p[1][e])  # noqa: E731
        rows = torch.from_numpy(t).to(x.device)
        h = torch.einsum("md,fd->mf", x[rows], _exact_weight(one(s["w_in"])))
        F = h.shape[1] // 2
        h = h[:, :F] / (1 + torch.exp(-h[:, :F])) * h[:, F:]
        part = torch.einsum("mf,df->md", h, _exact_weight(one(s["w_out"])))
        y[rows] += part * torch.from_numpy(w[t, j]).to(x.device).unsqueeze(1)
    return {"y": y, "ids": torch.from_numpy(ids.astype(np.int32)), "weights": torch.from_numpy(w)}


def _exact_verify(s):
    host, u = s["cu"][1], s["u"].double().cpu().numpy()
    tokens = s["tokens"].cpu().numpy()
    out, accepted = np.full(int(host[-1]), -1, np.int32), np.zeros(len(host) - 1, np.int32)
    for n in range(len(host) - 1):
        a, b = int(host[n]), int(host[n + 1])
        if a == b:
            continue
        i = a
        while i < b - 1:
            p = float(s["target"][i, tokens[i]])
            q = 1.0 if s["draft"] is None else float(s["draft"][i, tokens[i]])
            if not u[i] * q < p:
                break
            i += 1
        out[a:i] = tokens[a:i]
        rest = s["target"][i].double()
        if i < b - 1:
            if s["draft"] is None:
                rest[int(tokens[i])] = 0
            else:
                rest = torch.maximum(rest - s["draft"][i].double(), torch.zeros((), dtype=torch.float64, device=rest.device))
        cum = torch.cumsum(rest, 0)
        out[i] = int(torch.searchsorted(cum, cum[-1] * float(u[b - 1]), right=True))
        accepted[n] = i - a
    return {"tokens": torch.from_numpy(out), "accepted": torch.from_numpy(accepted)}


def exact(case, seed):
    s = prepare(case, seed)
    return {"gemm4": _exact_gemm4, "moe": _exact_moe, "verify": _exact_verify}[case["op"]](s)
