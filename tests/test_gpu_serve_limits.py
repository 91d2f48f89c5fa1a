"""4-bit weights, the mixture of experts and the verification of drafts at the limits of what they accept: largest batches,
magnitudes at either end, values that are not finite, kernels that take seconds."""
import numpy as np
import pytest
import torch

import kimi_delta_attention_16_gb300 as kda
import serve_testlib as lib
from serve_testlib import U, f64, gen, randn, within

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


def cuda(w):
    return w.cuda() if isinstance(w, torch.Tensor) else tuple(t.cuda() for t in w)


def experts(g, E, D, F, fmt, group=32, sdt=BF16):
    """Router, w_in, w_out on the GPU and the weights' values."""
    router = randn(g, E, D, std=D ** -0.5, dtype=BF16)
    if fmt == "bf16":
        wi, wo = randn(g, E, 2 * F, D, std=D ** -0.5, dtype=BF16), randn(g, E, D, F, std=F ** -0.5, dtype=BF16)
        return router, cuda(wi), cuda(wo), f64(wi), f64(wo)
    wi = lib.random_weight(g, E, 2 * F, D, fmt=fmt, group=group, scale_dtype=sdt)
    wo = lib.random_weight(g, E, D, F, fmt=fmt, group=group, scale_dtype=sdt)
    return router, cuda(wi), cuda(wo), lib.unpack_ref(*wi), lib.unpack_ref(*wo)


# ------------------------------------------------------------------ waits and their deadlines
def test_moe_first_products_longer_than_a_deadline():
    """The second products start beside the first ones and wait for them for as long as they take: 61,440 tokens that digits
    do not hold are multiplied one by one by a single CTA, for longer than a wait inside a kernel may last."""
    M, D, F = 65535, 2048, 32
    g = gen(50)
    router, wi, wo, wi64, wo64 = experts(g, 1, D, F, "e2m1")
    x = torch.full((M, D), 2.0 ** -110, dtype=BF16, device="cuda")
    some = torch.arange(0, M, 16)
    rows = randn(g, len(some), D, dtype=BF16)
    x[some.cuda()] = rows.cuda()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    y = kda.kda_moe(x, router.cuda(), wi, wo, 1, out_dtype=F32, d_status=status)
    assert int(status) == 0
    few = torch.arange(0, len(some), 400)
    ry, _, _, bound = lib.moe_ref(rows[few], router, wi64, wo64, 1, None, "sigmoid", 1.0)
    within(y[some[few].cuda()], ry, bound + U[F32] * (ry.abs() + bound))
    # what such a token's hidden values (|x|^2 and less) give lies below fp32's smallest
    rest = torch.ones(M, dtype=torch.bool)
    rest[some] = False
    assert bool((y[rest.cuda()] == 0).all())


def milliseconds(f, n=3):
    f()
    a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    torch.cuda.synchronize()
    a.record()
    for _ in range(n):
        f()
    b.record()
    torch.cuda.synchronize()
    return a.elapsed_time(b) / n


@pytest.mark.parametrize("fmt", ["e2m1", "int4", "bf16"])
def test_moe_many_tokens_of_nan(fmt):
    """Tokens whose logits are NaN all go to the lowest experts.  They leave the others' bits alone, and nothing is computed for
    them one by one: without such work the call takes two or three times as long at most (one expert in place of four has
    most of the tokens), with it some hundred times."""
    M, E, top, D, F = 2000, 16, 4, 1024, 256
    g = gen(51)
    router, wi, wo, _, _ = experts(g, E, D, F, fmt)
    router = router.cuda()
    x = randn(g, M, D, dtype=BF16).cuda()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    call = lambda: kda.kda_moe(x, router, wi, wo, top, out_dtype=F32, return_routing=True, d_status=status)  # noqa: E731
    clean, before = call(), milliseconds(call)
    x[::2, 5] = float("nan")
    y, ids, w = call()
    assert int(status) == 0
    assert bool(torch.isnan(y[::2]).all()) and bool(torch.isnan(w[::2]).all())
    assert torch.equal(ids[::2].cpu(), torch.arange(top, dtype=torch.int32).expand(M // 2, top))
    for a, b in zip(clean, (y, ids, w)):
        assert torch.equal(a[1::2], b[1::2])
    assert milliseconds(call) < 10 * before


# ------------------------------------------------------------------ magnitudes
@pytest.mark.parametrize("group,sdt", [(32, F32), (64, BF16), (128, F32)])
@pytest.mark.parametrize("exponent", [121, 122, 124, 126, 127])
def test_gemm4_integer_codes_largest_rows(group, sdt, exponent):
    """Rows that no power of two brings to where fp16 holds them are multiplied one by one; the result fits fp32, a code times x
    does not.  Each product is rounded twice (the eighth of a weight, the sum), which is less than what gemm4_ref allows."""
    M, N, K = 5, 60, 512
    g = gen(exponent + group)
    codes, scales = lib.random_weight(g, N, K, fmt="int4", group=group, scale_dtype=sdt, std=2.0 ** -30)
    x = torch.where(torch.rand(M, K, generator=g) < 0.5, -1.0, 1.0) * 2.0 ** exponent * (1 + 0.75 * torch.rand(M, K, generator=g)).clamp(max=1.75)
    x[3] = randn(g, K)  # beside an ordinary one
    x = x.to(BF16)
    got = kda.kda_gemm4(x.cuda(), codes.cuda(), scales.cuda(), out_dtype=F32)
    ref, err = lib.gemm4_ref(x, lib.unpack_ref(codes, scales), "none")
    assert float(ref.abs().max()) < 3e38
    # K products and as many additions, each within 2^-24 of the sum of magnitudes so far
    mass = f64(x).abs() @ lib.unpack_ref(codes, scales).abs().T
    within(got, ref, torch.maximum(err, (K + 2) * 2.0 ** -24 * mass) + U[F32] * ref.abs())


@pytest.mark.parametrize("sdt", [F32, BF16])
@pytest.mark.parametrize("M", [1, 20])
def test_gemm4_integer_codes_largest_scales(M, sdt):
    """Scales next to the end of fp32 (as kda_pack4 makes them of weights of 3e38) and small rows: a run's sum times its scale
    passes fp32 before the row's power of two is taken off, the result does not."""
    N, K = 40, 512
    g = gen(M)
    codes = torch.full((N, K // 2), 0xff, dtype=torch.uint8)
    codes[::4] = 0
    codes[1::4] = torch.randint(0, 256, codes[1::4].shape, generator=g, dtype=torch.uint8)
    scales = torch.full((N, K // 128), 4.5e37).to(sdt)
    x = (1e-10 * (1 + torch.rand(M, K, generator=g))).to(BF16)
    got = kda.kda_gemm4(x.cuda(), codes.cuda(), scales.cuda(), out_dtype=F32)
    w = lib.unpack_ref(codes, scales)
    ref, err = lib.gemm4_ref(x, w, "none")
    # or K products of an eighth of the weight, each with two roundings, added up one by one
    within(got, ref, torch.maximum(err, (K + 2) * 2.0 ** -24 * (f64(x).abs() @ w.abs().T)) + U[F32] * ref.abs())


@pytest.mark.parametrize("which", ["in", "out"])
def test_moe_integer_codes_largest_scales(which):
    """The same in either of the experts' products: x and, in the second, the weights of the first bring the values back."""
    M, E, top, D, F = 5, 3, 2, 256, 384
    g = gen(60)
    router, wi, wo, _, _ = experts(g, E, D, F, "int4", 128, F32)
    # the first products' weights are not negative, so that hidden values are of one sign
    wi[0].bitwise_or_(0x88)
    if which == "in":
        wi[0].fill_(0xff)
        wi[1].fill_(4.5e37)
        wo[1].mul_(1e-20)
    else:
        wo[0].fill_(0xff)
        wo[1].fill_(4.8e37)
    # gates and their counterparts of 1e8 and weights of 1e-22 behind them, or hidden values of 1e-26 and weights of 3e38
    x = (1 + torch.rand(M, D, generator=g)) * (1e-33 if which == "in" else 1e-13)
    x = x.to(BF16)
    y = kda.kda_moe(x.cuda(), router.cuda(), wi, wo, top, out_dtype=F32, score="softmax")
    wi64, wo64 = lib.unpack_ref(*wi), lib.unpack_ref(*wo)
    ry, _, _, bound = lib.moe_ref(x, router, wi64, wo64, top, None, "softmax", 1.0)
    assert 1e-6 < float(ry.abs().max()) < 1e30
    # products added up one by one instead of by groups: F + 2 roundings each of 2^-24 of the sum of magnitudes, where
    # moe_ref counts F / 32 + 16 of 2^-23 (for all of them at once: (F + 2) / 2 / (F / 32 + 16) = 6.9 times, D alike)
    within(y, ry, 8 * bound + U[F32] * ry.abs())


@pytest.mark.parametrize("M,dtype", [(1, F32), (7, BF16), (40, F32), (130, BF16)])
def test_gemm4_e2m1_results_next_to_the_end_of_fp32(M, dtype):
    """1.75 times 2^127 is 2.98e38; its digit in front, 2 times 2^127, is not a number of fp32.  Rows that hold it alone, exact, and
    beside others that do overflow."""
    N, K = 30, 64
    codes = torch.zeros(N, K // 2, dtype=torch.uint8)
    codes[:, 5] = 2  # 1.0 at element 10
    codes[1::2, 5] = 10  # -1.0
    codes[2, 5] = 6  # 4.0
    codes[:, 20] = 2  # and 1.0 at element 40
    scales = torch.full((N, K // 32), 254, dtype=torch.uint8)
    scales[:, 1] = 127
    x = torch.zeros(M, K)
    x[:, 10] = 1.75
    x[:, 40] = 2.0 ** 110  # lies below a bf16's last digit of the first, above an fp32's
    got = kda.kda_gemm4(x.to(BF16).cuda(), codes.cuda(), scales.cuda(), out_dtype=dtype)
    want = (x.double() @ lib.unpack_ref(codes, scales).T).float()
    assert bool(torch.isinf(want[:, 2]).all()) and int(torch.isinf(want).sum()) == M
    assert torch.equal(got.cpu(), want.to(dtype))


def test_moe_e2m1_gates_next_to_the_end_of_fp32():
    """The same in the experts' first products: a gate of -2.98e38 gives a hidden value of 0, one that overflows as well; a gate of
    2.98e38 under a counterpart of 1e-38 an ordinary one."""
    E, D, F = 2, 64, 32
    ci, si = torch.zeros(E, 2 * F, D // 2, dtype=torch.uint8), torch.full((E, 2 * F, D // 32), 127, dtype=torch.uint8)
    ci[:, :F, 0] = 2   # gates: x[0] 2^127
    ci[:, :F // 2, 0] = 10
    si[:, :F, 0] = 254
    ci[:, F:, 16] = 2  # the other side: x[32] 2^-126
    si[:, F:, 1] = 1
    g = gen(70)
    wo = lib.random_weight(g, E, D, F, fmt="e2m1", group=32)
    x = torch.zeros(3, D)
    x[:, 0], x[:, 32] = 1.75, 1.0
    router = randn(g, E, D, dtype=BF16)
    y = kda.kda_moe(x.to(BF16).cuda(), router.cuda(), (ci.cuda(), si.cuda()), cuda(wo), 2, out_dtype=F32, score="softmax")
    h = torch.zeros(F, dtype=torch.float64)
    h[F // 2:] = 1.75 * 2.0  # silu(1.75 2^127) 2^-126
    w = torch.softmax(x.double() @ f64(router).T, 1)
    parts = torch.stack([lib.unpack_ref(wo[0][e], wo[1][e]) @ h for e in range(E)])
    # a hidden value and a weight, each rounded once, products exact, F additions
    mass = torch.stack([lib.unpack_ref(wo[0][e], wo[1][e]).abs() @ h for e in range(E)])
    within(y, w @ parts, (F + 8) * 2.0 ** -24 * (w @ mass))


@pytest.mark.parametrize("M", [100, 130])
@pytest.mark.parametrize("K", [12288, 32768, 40000, 131072, 262144, 294912])
def test_gemm4_many_rows_do_not_shrink(M, K):
    """Long sums of products of one sign, more than 96 rows and a bf16 result, on as many tiles as there are SMs (so that no
    cluster shares K of its own accord): an accumulator takes 32,768 elements, 2,048 instructions that cut off 2^-23 of what
    has come together so far, half of the sum on average: 2^-13 for all results together at most, whatever the length.
    Rounding to bf16 leaves nothing of the kind: the results spread evenly over a power of two, each is off by 2^-8 / sqrt(12) of
    itself on average, so all 1.9 million of them by 6 * 2^-8 / sqrt(12 * 1.9e6) = 5e-6 together (six standard deviations)."""
    N = 128 * 152
    g = torch.Generator(device="cuda")
    g.manual_seed(K + M)
    codes = torch.randint(0, 256, (N, K // 2), generator=g, device="cuda", dtype=torch.uint8) & 0x77  # 0 to 6
    # the first part of a row's scales a power of two lower, so that rows differ by up to 2
    scales = torch.full((N, K // 32), 120, device="cuda", dtype=torch.uint8)
    share = torch.rand(N, 1, generator=g, device="cuda")
    scales -= (torch.arange(K // 32, device="cuda").unsqueeze(0) < share * (K // 32)).to(torch.uint8)
    x = (torch.rand(M, K, generator=g, device="cuda") * (1 + torch.rand(M, 1, generator=g, device="cuda"))).to(BF16)
    y = kda.kda_gemm4(x, codes, scales).double()
    ref = kda.kda_gemm4(x, codes, scales, out_dtype=F32).double()  # rounded sums, 1e-7 off
    assert abs(float((y / ref - 1).mean())) < 2.0 ** -13 + 5e-6
    assert float((y / ref - 1).abs().max()) < 2.0 ** -12 + 2.0 ** -8


def test_gemm4_many_rows_tiny_values():
    """Rows of any magnitude beside one another, from 97 rows on as below: products and sums that fp32 holds as subnormal numbers only
    are kept."""
    N, K = 70, 640
    g = gen(80)
    codes, scales = lib.random_weight(g, N, K, fmt="e2m1", group=32)
    for M in (96, 97, 140, 260):
        x = randn(g, M, K)
        x[1] = 0
        x *= 2.0 ** torch.arange(0, -M, -1).clamp(min=-122).float().unsqueeze(1)
        x[5, 32:64] *= 2.0 ** -100
        x = x.to(BF16)
        got = kda.kda_gemm4(x.cuda(), codes.cuda(), scales.cuda())
        ref, err = lib.gemm4_ref(x, lib.unpack_ref(codes, scales), "none")
        # the result's last digit is 2^-133 at least, an fp32 sum's 2^-149
        within(got, ref, torch.maximum(err, torch.tensor(K * 2.0 ** -149)) + torch.maximum(U[BF16] * (ref.abs() + err), torch.tensor(2.0 ** -134)))


# ------------------------------------------------------------------ verification
def one_draft(p, q, u):
    """Whether the draft of token 0 stands, for every triple: sequences of two rows over two tokens."""
    n = len(u)
    target, draft = torch.ones(2 * n, 2), torch.ones(2 * n, 2)
    target[::2, 0], draft[::2, 0] = p, q
    us = torch.full((2 * n,), 0.25)
    us[::2] = u
    cu = np.arange(0, 2 * n + 1, 2, dtype=np.int32)
    out, accepted = kda.kda_verify(target.cuda(), torch.zeros(2 * n, dtype=torch.int32).cuda(), us.cuda(), cu, draft=draft.cuda())
    assert bool(((out.cpu()[::2] == 0) | (accepted.cpu() == 0)).all())
    return accepted.cpu().bool()


def positive(v):
    return torch.where(v > 0, v, torch.zeros_like(v)).double()


def test_verify_drafts_of_any_value():
    """Values that are not above 0 count as 0 on both sides; products of the smallest and of neighbours are not rounded."""
    nan = float("nan")
    vs = [nan, -1.0, -0.5, -1e-40, -0.0, 0.0, 1e-45, 3e-39, 2.0 ** -61, 2.0 ** -60, 0.1, 0.5, 1.0 - 2.0 ** -24, 1.0]
    us = [0.0, 1e-45, 2.0 ** -64, 2.0 ** -24, 0.1, 0.5, 1.0 - 2.0 ** -24]
    p, q, u = (t.reshape(-1).float() for t in torch.meshgrid(torch.tensor(vs), torch.tensor(vs), torch.tensor(us), indexing="ij"))
    want = u.double() * positive(q) < positive(p)  # exact: 48 bits
    assert torch.equal(one_draft(p, q, u), want)


def test_verify_large_values_beside_small_ones():
    """Values need not sum to 1: a draft's value from 2^64 on beside a target's below 2^-60, u of 0 among them."""
    vs = [1e-45, 1e-39, 1e-20, 2.0 ** -61, 2.0 ** -60, 1.0, 2.0 ** 63, 2.0 ** 64, 1e30, 3e38]
    us = [0.0, 1e-45, 1e-38, 2.0 ** -64, 0.5]
    p, q, u = (t.reshape(-1).float() for t in torch.meshgrid(torch.tensor(vs), torch.tensor(vs), torch.tensor(us), indexing="ij"))
    assert torch.equal(one_draft(p, q, u), u.double() * q.double() < p.double())


@pytest.mark.parametrize("V", [50, 5000, 40001])
@pytest.mark.parametrize("N", [1, 200])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_verify_infinities_draw_nothing(N, V, dtype):
    """What is drawn from with an infinity in it, or a sum beyond fp32, gives -1 wherever it stands and whatever u is; the other sequences
    are as they were."""
    g = gen(V + N)
    inf = float("inf")
    p = torch.rand(2 * N, V, generator=g).to(dtype)
    q = torch.rand(2 * N, V, generator=g).to(dtype)
    p[::2, 0], q[::2, 0] = 0.25, 0.5  # token 0 is proposed: taken where u is below a half
    u = torch.rand(2 * N, generator=g)
    tokens, cu = torch.zeros(2 * N, dtype=torch.int32), np.arange(0, 2 * N + 1, 2, dtype=np.int32)
    run = lambda p, q: [t.cpu() for t in kda.kda_verify(p.cuda(), tokens.cuda(), u.cuda(), cu, draft=None if q is None else q.cuda())]  # noqa: E731
    for at in (1, V // 2, V - 1):
        for where, value in ((p, inf), (q, inf), (p, 3.0e38)):
            a, b = p.clone(), q.clone()
            bad = a if where is p else b
            bad[::6, at] = value       # the first of two rows: what is drawn from after a refusal
            bad[1::6, at] = value      # the second: after an acceptance
            if value < inf:
                bad[::6, 2], bad[1::6, 2] = 3.0e38, 3.0e38  # two of them: their sum, or the rest of it, passes fp32
                if at == 2:
                    continue
            for draft in (b, None):
                plain, (out, accepted) = run(p, None if draft is None else q), run(a, draft)
                assert torch.equal(accepted, plain[1])
                for n in range(N):
                    row = 2 * n + int(accepted[n])
                    if n % 3 == 0 and not (where is q and (draft is None or accepted[n])):
                        assert int(out[row]) == -1
                        out[row] = plain[0][row]
                assert torch.equal(out, plain[0])


# ------------------------------------------------------------------ one workspace, call after call
@pytest.mark.parametrize("fmt", ["e2m1", "bf16", "int4"])
def test_moe_one_workspace_other_experts_every_call(fmt):
    """Calls in a row in one workspace, eager and replayed: each reads the lists of its own tokens, not what the call in front left
    in the same place."""
    M, E, top, D, F, n = 6, 60, 3, 256, 128, 8
    g = gen(90)
    router, wi, wo, _, _ = experts(g, E, D, F, fmt)
    router = (4 * router.float()).to(BF16).cuda()
    xs = [randn(g, M, D, dtype=BF16).cuda() for _ in range(n)]
    call = lambda x, **kw: kda.kda_moe(x, router, wi, wo, top, return_routing=True, **kw)  # noqa: E731
    want = [call(x) for x in xs]
    assert len({tuple(w[1].flatten().tolist()) for w in want}) == n
    ws = torch.zeros(1 << 22, dtype=torch.uint8, device="cuda")
    held = [x.clone() for x in xs]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = [call(x, workspace=ws) for x in held]
    for turn in range(12):
        order = [(i * (1 + 2 * (turn % 4)) + turn) % n for i in range(n)]
        for h, i in zip(held, order):
            h.copy_(xs[i])
        graph.replay()
        eager = [call(xs[i], workspace=ws) for i in order]
        for outs in (got, eager):
            for o, i in zip(outs, order):
                assert all(torch.equal(a, b) for a, b in zip(o, want[i]))


@pytest.mark.parametrize("fmt,floor", [("e2m1", 2.0 ** -127), ("int4", 0.0), ("bf16", 2.0 ** -134)])
@pytest.mark.parametrize("exponent", [-120, -90, -75, -60, -57, -54, -50, -40, -20, 0, 20, 40, 55])
def test_moe_magnitudes(exponent, fmt, floor):
    """Tokens of any magnitude: hidden values of about its square, of which what lies below `floor` may be dropped."""
    M, E, top, D, F = 4, 6, 2, 128, 96
    g = gen(100)
    router, wi, wo, wi64, wo64 = experts(g, E, D, F, fmt)
    x = (randn(g, M, D) * 2.0 ** exponent).to(BF16)
    logits = f64(x) @ f64(router).T
    for score in ("softmax", "sigmoid"):
        y, ids, w = kda.kda_moe(x.cuda(), router.cuda(), wi, wo, top, out_dtype=F32, score=score, return_routing=True)
        ids = ids.cpu().long()
        # no expert that was left out has a score that is larger by more than 2^-50 (a logit by 2^-48 where it is small)
        out = logits.clone().scatter_(1, ids, -torch.inf)
        best, worst = (torch.sigmoid(v) if score == "sigmoid" else v for v in (out.amax(1), logits.gather(1, ids).amin(1)))
        assert bool((best <= worst + (2.0 ** -50 if score == "sigmoid" else 0.0)).all())
        # the reference for this choice: a bias that makes it
        for t in range(M):
            choice = torch.full((E,), -9.0 if score == "sigmoid" else -torch.inf).index_fill_(0, ids[t], 0.0)
            if score == "sigmoid":
                ry, rids, rw, bound = lib.moe_ref(x[t:t + 1], router, wi64, wo64, top, choice, score, 1.0)
            else:
                ry, rids, rw, bound = lib.moe_ref(x[t:t + 1], router, wi64, wo64, top, None, score, 1.0)
            assert sorted(rids[0].tolist()) == sorted(ids[t].tolist())
            # the floor and, of gates, hidden values, products and sums, the last digit of fp32's subnormal numbers
            hidden = floor + 4 * 2.0 ** -149
            small = sum(rw[0, j] * (wo64[rids[0, j]].abs().sum(1) * hidden + (F + 4) * 2.0 ** -149) for j in range(top))
            within(y[t:t + 1], ry, bound + U[F32] * (ry.abs() + bound) + small, score)


@pytest.mark.parametrize("with_bias", [False, True])
def test_moe_scores_around_a_half(with_bias):
    """Scores that 53 bits do not tell apart are equal, whichever sign their logits have, and go to the lower expert; small logits
    that they do tell apart are chosen by."""
    M, E, top, D, F = 8, 40, 5, 64, 32
    g = gen(110)
    router, wi, wo, _, _ = experts(g, E, D, F, "e2m1")
    bias = torch.zeros(E).cuda() if with_bias else None
    for exponent in (-120, -100, -70, -60, -40, -30, -25, -20, -15, -10):
        x = (randn(g, M, D) * 2.0 ** exponent).to(BF16)
        _, ids, _ = kda.kda_moe(x.cuda(), router.cuda(), wi, wo, top, bias=bias, return_routing=True)
        key = f64(x) @ f64(router).T if exponent >= -40 else torch.zeros(M, E, dtype=torch.float64)
        want = torch.sort(key, dim=1, descending=True, stable=True).indices[:, :top]
        assert torch.equal(ids.cpu().long(), want), exponent


# ------------------------------------------------------------------ the largest batches
@pytest.mark.parametrize("fmt,group,sdt", lib.FORMATS)
@pytest.mark.parametrize("out_dtype", [F32, BF16])
@pytest.mark.parametrize("M", [1001, 5000, 65535])
def test_gemm4_largest_batches(M, fmt, group, sdt, out_dtype):
    N, K = 70, 384
    g = gen(M)
    x = randn(g, M, K, dtype=BF16)
    codes, scales = lib.random_weight(g, N, K, fmt=fmt, group=group, scale_dtype=sdt)
    got = kda.kda_gemm4(x.cuda(), codes.cuda(), scales.cuda(), out_dtype=out_dtype)
    ref, err = lib.gemm4_ref(x, lib.unpack_ref(codes, scales), "none")
    within(got, ref, err + U[out_dtype] * (ref.abs() + err))


def moe_ref_by_expert(x, router, w_in, w_out, ids, w):
    """serve_testlib.moe_ref's y and bound for a given choice and its weights, an expert's tokens at a time on the GPU."""
    x, w_in, w_out, ids = f64(x).cuda(), w_in.cuda(), w_out.cuda(), ids.long().cuda()
    w = w.double().cuda()
    D, F = w_out.shape[1], w_out.shape[2]
    y, bound = torch.zeros_like(x), torch.zeros_like(x)
    for e in range(w_in.shape[0]):
        t, j = torch.nonzero(ids == e, as_tuple=True)
        if not len(t):
            continue
        gu, dgu = x[t] @ w_in[e].T, (D / 32 + 16) * 2.0 ** -23 * (x[t].abs() @ w_in[e].abs().T)
        gate, u, dg, du = gu[:, :F], gu[:, F:], dgu[:, :F], dgu[:, F:]
        s = gate * torch.sigmoid(gate)
        h = s * u
        dh = 1.1 * dg * (u.abs() + du) + s.abs() * du + 12 * 2.0 ** -24 * h.abs() + 2.0 ** -21 * h.abs() + 2.0 ** -36 * h.abs().amax(1, keepdim=True)
        p = h @ w_out[e].T
        dp = dh @ w_out[e].abs().T + (F / 32 + 16) * 2.0 ** -23 * ((h.abs() + dh) @ w_out[e].abs().T)
        k = w[t, j].unsqueeze(1)
        y.index_add_(0, t, k * p)  # a token has an expert once
        bound.index_add_(0, t, k * (dp + 8 * 2.0 ** -24 * p.abs()))
    return y, bound + ids.shape[1] * 2.0 ** -23 * y.abs()


@pytest.mark.parametrize("fmt", ["e2m1", "int4", "bf16"])
@pytest.mark.parametrize("M,E,top", [(65535, 5, 1), (2047, 1024, 32), (8191, 64, 8), (300, 200, 6)])
def test_moe_largest_batches(M, E, top, fmt):
    """Up to 65,535 places of tokens with experts: slots, lists and their 16-bit starts, many passes over an expert's tokens."""
    D, F = 128, 96
    g = gen(M)
    router, wi, wo, wi64, wo64 = experts(g, E, D, F, fmt)
    x = randn(g, M, D, dtype=BF16)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    y, ids, w = kda.kda_moe(x.cuda(), router.cuda(), wi, wo, top, score="softmax", scale=1.5, out_dtype=F32, return_routing=True, d_status=status)
    assert int(status) == 0
    logits = f64(x) @ f64(router).T
    want = torch.sort(logits, dim=1, descending=True, stable=True)
    assert torch.equal(ids.cpu().long(), want.indices[:, :top])
    rw = 1.5 * torch.softmax(want.values[:, :top], 1)
    within(w, rw, 2.0 ** -23 * rw)
    ry, bound = moe_ref_by_expert(x, router, wi64, wo64, ids, rw)
    within(y, ry.cpu(), (bound + U[F32] * (ry.abs() + bound)).cpu())


# ------------------------------------------------------------------ one large value beside small ones
@pytest.mark.parametrize("M", [5, 130])
def test_gemm4_e2m1_large_value_beside_small_ones(M):
    """A value holds what lies above 2^-22 of the largest of its 32, however small that one's weight is: the largest of a group has a
    weight of 0, the others are 1 to 2 and 2^6 to 2^24 times smaller.  From 97 rows on with a bf16 result nothing is lost."""
    N, K = 60, 256
    g = gen(120)
    codes, scales = lib.random_weight(g, N, K, fmt="e2m1", group=32)
    codes[:, ::16] &= 0xf0  # element 0 of each group
    w = lib.unpack_ref(codes, scales)
    for exponent in (6, 14, 18, 22, 24):
        x = 1 + torch.rand(M, K, generator=g)
        x[:, ::32] = 2.0 ** exponent
        x = x.to(BF16)
        for dtype in (BF16, F32):
            got = kda.kda_gemm4(x.cuda(), codes.cuda(), scales.cuda(), out_dtype=dtype)
            ref, err = lib.gemm4_ref(x, w, "none")
            # bf16 values of 1 to 2 end at 2^-7: exact where that is above 2^-22 of the largest
            lost = 0.0 if exponent <= 14 or (M > 96 and dtype is BF16) else 2.0 ** (exponent - 22)
            within(got, ref, err + lost * w.abs().sum(1) + U[dtype] * (ref.abs() + err), f"{exponent} {dtype}")


# ------------------------------------------------------------------ the largest sizes
@pytest.mark.parametrize("fmt,group,sdt", lib.FORMATS)
@pytest.mark.parametrize("M", [2, 100])
def test_gemm4_longest_rows(M, fmt, group, sdt):
    """Rows of 2^24 weights, of which few meet an x that is not 0: the others, and the groups' sums that they leave, add nothing."""
    N, K = 3, 1 << 24
    g = torch.Generator(device="cuda")
    g.manual_seed(M)
    codes = torch.randint(0, 256, (N, K // 2), generator=g, device="cuda", dtype=torch.uint8)
    scales = torch.full((N, K // group), 118, device="cuda", dtype=torch.uint8) if fmt == "e2m1" else torch.full((N, K // group), 0.25, device="cuda", dtype=sdt)
    at = torch.cat([torch.randint(0, K, (60,), generator=g, device="cuda"), torch.tensor([0, K - 1], device="cuda")]).unique()
    x = torch.zeros(M, K, dtype=BF16, device="cuda")
    x[:, at] = torch.randn(M, len(at), generator=g, device="cuda").to(BF16)
    got = kda.kda_gemm4(x, codes, scales, out_dtype=F32)
    c = (codes[:, at // 2].int() >> (4 * (at % 2)).int()) & 15
    w = torch.cat([lib.E2M1, -lib.E2M1]).cuda()[c.long()] * 2.0 ** -9 if fmt == "e2m1" else (c - 8).double() * 0.25
    ref, mass = x[:, at].double() @ w.T, x[:, at].double().abs() @ w.abs().T
    # a term's own rounding, and (integer codes) those of the 8 that is taken off its group's sum: 80 roundings of a group's
    # 8 |x| at most
    extra = 0.0 if fmt == "e2m1" else 80 * 2.0 ** -23 * 0.25 * 8 * x[:, at].double().abs().sum(1, keepdim=True)
    within(got, ref.cpu(), (80 * 2.0 ** -23 * mass + extra).cpu())


@pytest.mark.parametrize("fmt,sdt", [("e2m1", torch.uint8), ("int4", F32)])
def test_gemm4_most_outputs(fmt, sdt):
    N, K, M = 1 << 24, 32, 3
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    codes = torch.randint(0, 256, (N, K // 2), generator=g, device="cuda", dtype=torch.uint8)
    scales = torch.randint(118, 126, (N, 1), generator=g, device="cuda").to(torch.uint8) if fmt == "e2m1" else torch.rand(N, 1, generator=g, device="cuda") + 0.1
    x = torch.randn(M, K, generator=g, device="cuda").to(BF16)
    got = kda.kda_gemm4(x, codes, scales, out_dtype=F32)
    assert bool(torch.isfinite(got).all())
    some = torch.cat([torch.arange(1000), torch.randint(0, N, (4000,), generator=gen(2)), torch.arange(N - 1000, N)])
    ref, err = lib.gemm4_ref(x, lib.unpack_ref(codes[some.cuda()], scales[some.cuda()]), "none")
    within(got[:, some.cuda()], ref, err + U[F32] * ref.abs())


@pytest.mark.parametrize("N", [1, 40, 304])
def test_verify_largest_vocabulary(N):
    """4,000,000 tokens, by one CTA of a row or by eight."""
    V = 4000000
    p = torch.rand(N, V, device="cuda").to(BF16)
    u = torch.rand(N, generator=gen(N))
    out, _ = kda.kda_verify(p, torch.zeros(N, dtype=torch.int64).cuda(), u.cuda(), np.arange(N + 1, dtype=np.int32))
    for n in {0, N // 2, N - 1}:
        ro, _ = lib.verify_ref(p[n:n + 1].cpu(), None, torch.zeros(1, dtype=torch.int64), u[n:n + 1], np.array([0, 1], np.int32))
        assert int(out[n]) == int(ro[0])


def test_verify_long_and_many_sequences():
    """A hundred thousand drafts of a sequence, all taken or none; two hundred thousand sequences."""
    V, lens = 9, [100000, 1, 0, 50000, 70001]
    T = sum(lens)
    g = gen(3)
    p, u = torch.rand(T, V, generator=g) + 0.1, torch.rand(T, generator=g) * 0.5
    tokens = torch.randint(0, V, (T,), generator=g).int()
    q = p.clone()
    first = 150001  # of the last sequence, which stops at 60,000
    q[first + 60000, tokens[first + 60000]] = 50.0
    u[first + 60000] = 0.9
    cu = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
    out, accepted = kda.kda_verify(p.cuda(), tokens.cuda(), u.cuda(), cu, draft=q.cuda())
    assert accepted.tolist() == [99999, 0, 0, 49999, 60000]
    out = out.cpu()
    for n, a in enumerate(accepted.tolist()):
        b = int(cu[n])
        assert torch.equal(out[b:b + a], tokens[b:b + a]) and bool((out[b + a + 1:int(cu[n + 1])] == -1).all())
    n = 200000
    p, u = torch.rand(n, V, generator=g), torch.rand(n, generator=g)
    out, accepted = kda.kda_verify(p.cuda(), torch.zeros(n, dtype=torch.int32).cuda(), u.cuda(), np.arange(n + 1, dtype=np.int32))
    cum = p.double().cumsum(1)
    assert torch.equal(out.cpu().long(), (cum > u.double().unsqueeze(1) * cum[:, -1:]).int().argmax(1)) and not bool(accepted.any())


@pytest.mark.parametrize("fmt", ["e2m1", "int4", "bf16"])
def test_moe_smallest_and_widest(fmt):
    """Experts of the least sizes, and rows of 2^17 and more on either side."""
    unit = 8 if fmt == "bf16" else 32
    for M, E, top, D, F in ((3, 4, 2, unit, unit), (1, 1, 1, unit, 96), (2, 2, 1, (1 << 17) + 96, 32), (2, 2, 2, 64, (1 << 17) + 32)):
        g = gen(D + F)
        router, wi, wo, wi64, wo64 = experts(g, E, D, F, fmt)
        x = randn(g, M, D, dtype=BF16)
        y, ids, w = kda.kda_moe(x.cuda(), router.cuda(), wi, wo, top, out_dtype=F32, score="softmax", return_routing=True)
        ry, rids, rw, bound = lib.moe_ref(x, router, wi64, wo64, top, None, "softmax", 1.0)
        assert torch.equal(ids.cpu().long(), rids)
        within(y, ry, bound + U[F32] * (ry.abs() + bound), f"{D} x {F}")
