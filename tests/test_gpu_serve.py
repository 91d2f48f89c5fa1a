"""4-bit weights, the mixture of experts and the verification of drafts on the GPU against plain 64-bit forms."""
import numpy as np
import pytest
import torch

import kimi_delta_attention_16_gb300 as kda
import serve_testlib as lib
from serve_testlib import FORMATS, U, f64, gen, randn, within

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


def dev(*ts):
    out = tuple(t.cuda() if isinstance(t, torch.Tensor) else t for t in ts)
    return out if len(out) > 1 else out[0]


# ------------------------------------------------------------------ packing
@pytest.mark.parametrize("fmt,group,sdt", FORMATS)
@pytest.mark.parametrize("rows,K", [(1, 128), (7, 256), (300, 1152)])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_pack4_codes_and_scales(fmt, group, sdt, rows, K, dtype):
    g = gen(rows + K)
    w = randn(g, rows, K, dtype=dtype) * torch.exp(3 * torch.randn(rows, 1, generator=g)).to(dtype)
    w[0, :group] = 0
    w[-1, -1] = 1e-40 if dtype == F32 else 1e-38
    codes, scales = kda.kda_pack4(w.cuda(), format=fmt, group=group, scale_dtype=sdt or BF16)
    rc, rs = lib.pack_ref(w, fmt, group, sdt)
    assert scales.dtype == (torch.uint8 if fmt == "e2m1" else sdt)
    assert torch.equal(scales.cpu(), rs)
    got = torch.stack([codes & 15, codes >> 4], -1).view(rows, K).cpu().long()
    # a zero may carry either sign in e2m1
    same = (got == rc) | ((fmt == "e2m1") & ((got & 7) == 0) & ((rc & 7) == 0))
    assert bool(same.all())
    for dt in (BF16, F32):
        back = kda.kda_unpack4(codes, scales, dtype=dt)
        assert torch.equal(f64(back), f64(lib.unpack_ref(codes, scales).to(dt)))


def test_pack4_strided_and_leading_axes():
    w = randn(gen(5), 2, 3, 4, 192)
    codes, scales = kda.kda_pack4(w.cuda())
    assert codes.shape == (2, 3, 4, 96) and scales.shape == (2, 3, 4, 6)
    big = torch.zeros(24, 201, device="cuda")
    big[:, 3:195] = w.view(24, 192).cuda()
    c2, s2 = kda.kda_pack4(big[:, 3:195])  # rows that are not 16-byte aligned
    assert torch.equal(c2.view(-1), codes.view(-1)) and torch.equal(s2.view(-1), scales.view(-1))
    assert kda.kda_pack4(big[:0, 3:195])[0].shape == (0, 96)


# ------------------------------------------------------------------ gemm4
def check_gemm4(M, N, K, fmt, group, sdt, epilogue="none", out_dtype=None, seed=0, x=None):
    g = gen(seed + M + 3 * N + 7 * K)
    x = randn(g, M, K, dtype=BF16) if x is None else x
    codes, scales = lib.random_weight(g, N, K, fmt=fmt, group=group, scale_dtype=sdt)
    got = kda.kda_gemm4(x.cuda(), codes.cuda(), scales.cuda(), epilogue=epilogue, out_dtype=out_dtype)
    want = out_dtype or (BF16 if epilogue == "none" else F32)
    assert got.dtype == want and got.shape == (M, N)
    ref, err = lib.gemm4_ref(x, lib.unpack_ref(codes, scales), epilogue)
    within(got, ref, err + U[want] * (ref.abs() + err), f"{M}x{N}x{K} {fmt}/{group} {epilogue}")


@pytest.mark.parametrize("fmt,group,sdt", FORMATS)
@pytest.mark.parametrize("M,N,K", [(1, 1, 128), (1, 128, 256), (2, 129, 384), (8, 127, 1024), (9, 300, 1152), (16, 64, 2176),
                                   (17, 257, 1280), (33, 40, 640), (64, 130, 512), (65, 96, 384), (130, 200, 256)])
def test_gemm4_sizes(M, N, K, fmt, group, sdt):
    check_gemm4(M, N, K, fmt, group, sdt, out_dtype=F32)


@pytest.mark.parametrize("M", [1, 5, 12, 40])
@pytest.mark.parametrize("K", [32, 64, 96, 224, 288, 1056, 2080, 4128])
def test_gemm4_odd_groups(M, K):
    check_gemm4(M, 70, K, "e2m1", 32, None, out_dtype=F32)
    check_gemm4(M, 70, K, "int4", 32, F32)


@pytest.mark.parametrize("epilogue", ["none", "decay", "sigmoid"])
@pytest.mark.parametrize("out_dtype", [BF16, F32, None])
def test_gemm4_epilogues(epilogue, out_dtype):
    check_gemm4(5, 333, 1056, "int4", 32, BF16, epilogue, out_dtype)
    check_gemm4(20, 96, 7168, "e2m1", 32, None, epilogue, out_dtype)


def test_gemm4_many_tiles():
    check_gemm4(3, 20000, 512, "e2m1", 32, None)
    check_gemm4(70, 9000, 256, "int4", 128, BF16)


@pytest.mark.parametrize("fmt,group,sdt", FORMATS)
@pytest.mark.parametrize("exponent", [-120, -60, 0, 60, 100])
def test_gemm4_magnitudes(exponent, fmt, group, sdt):
    """Columns of any magnitude, and elements far below the largest of their run."""
    g = gen(exponent + 200)
    x = randn(g, 6, 1024) * torch.exp2(torch.randint(-25, 1, (6, 1024), generator=g).float()) * 2.0 ** exponent
    check_gemm4(6, 50, 1024, fmt, group, sdt, out_dtype=F32, x=x.to(BF16))


@pytest.mark.parametrize("fmt,group,sdt", FORMATS)
def test_gemm4_not_finite_stays_in_its_row(fmt, group, sdt):
    g = gen(3)
    x = randn(g, 4, 512, dtype=BF16)
    x[1, 300] = float("inf")
    x[2, 5] = float("nan")
    codes, scales = lib.random_weight(g, 60, 512, fmt=fmt, group=group, scale_dtype=sdt)
    got = kda.kda_gemm4(x.cuda(), codes.cuda(), scales.cuda(), out_dtype=F32).cpu()
    w = lib.unpack_ref(codes, scales)
    ref, err = lib.gemm4_ref(x[[0, 3]], w, "none")
    within(got[[0, 3]], ref, err + U[F32] * ref.abs())
    inf = torch.where(w[:, 300] == 0, torch.nan, torch.inf * w[:, 300].sign())
    assert torch.equal(torch.isnan(got[1]), torch.isnan(inf)) and torch.equal(got[1].nan_to_num(), inf.float().nan_to_num())
    assert bool(torch.isnan(got[2]).all())


def test_gemm4_rows_of_zeros_and_tiny_values():
    """Padding beside rows in use, rows whose values all lie below what digits hold, and such values beside others."""
    g = gen(14)
    x = randn(g, 5, 640)
    x[1] = 0
    x[2] *= 2.0 ** -115
    x[3, 32:64] *= 2.0 ** -110
    for fmt, group, sdt in FORMATS:
        check_gemm4(5, 60, 640, fmt, group, sdt, out_dtype=F32, x=x.to(BF16))


@pytest.mark.parametrize("fmt", ["e2m1", "int4"])
def test_gemm4_strides_and_alignment(fmt):
    g = gen(11)
    x = randn(g, 7, 300, dtype=BF16)
    codes, scales = lib.random_weight(g, 90, 288, fmt=fmt, group=32, scale_dtype=BF16)
    ref, err = lib.gemm4_ref(x[:, 5:293], lib.unpack_ref(codes, scales), "none")
    big = torch.full((7, 101), 7.0, device="cuda")
    out = kda.kda_gemm4(x.cuda()[:, 5:293], codes.cuda(), scales.cuda(), out=big[:, 3:93])
    assert out.data_ptr() == big[:, 3:].data_ptr()
    within(out, ref, err + U[F32] * ref.abs())
    assert bool((big[:, :3] == 7).all()) and bool((big[:, 93:] == 7).all())


@pytest.mark.parametrize("fmt,group,sdt", FORMATS)
def test_gemm4_empty_and_same_bits(fmt, group, sdt):
    g = gen(12)
    x = randn(g, 30, 2304, dtype=BF16).cuda()
    codes, scales = (t.cuda() for t in lib.random_weight(g, 500, 2304, fmt=fmt, group=group, scale_dtype=sdt))
    one = kda.kda_gemm4(x, codes, scales, out_dtype=F32)
    assert torch.equal(one, kda.kda_gemm4(x, codes, scales, out_dtype=F32))
    assert kda.kda_gemm4(x[:0], codes, scales).shape == (0, 500)
    assert kda.kda_gemm4(x, codes[:0], scales[:0]).shape == (30, 0)


@pytest.mark.parametrize("fmt,sdt", [("e2m1", torch.uint8), ("int4", F32)])
def test_gemm4_offsets_past_32_bits(fmt, sdt):
    """Codes of 4.6 GB: the last rows are at offsets that 32 bits do not hold."""
    N, K = 600000, 15360
    if torch.cuda.mem_get_info()[0] < 12 << 30:
        pytest.skip("needs 12 GB of free memory")
    codes = torch.full((N, K // 2), 0 if fmt == "e2m1" else 0x88, dtype=torch.uint8, device="cuda")  # weights of 0
    scales = torch.full((N, K // 32), 127 if fmt == "e2m1" else 1.0, dtype=sdt, device="cuda")
    g = gen(13)
    tail, st = lib.random_weight(g, 200, K, fmt=fmt, group=32, scale_dtype=sdt)
    codes[-200:], scales[-200:] = tail.cuda(), st.cuda()
    x = randn(g, 2, K, dtype=BF16)
    got = kda.kda_gemm4(x.cuda(), codes, scales, out_dtype=F32)
    # Integer codes enter as they are, and 8 times a group's sum of x is taken off: of a group of zeros (codes 8, scale 1)
    # remain the roundings of that sum (32 additions) and of the two matrix instructions that build it up again, each at
    # most 2^-23 of 8 sum |x|; groups add up, each addition within 2^-24 of what is left so far.
    zeros = 0.0 if fmt == "e2m1" else float(36 * 2.0 ** -23 * 8 * f64(x).abs().sum(1).max())
    assert bool((got[:, :-200].abs() <= zeros).all())
    ref, err = lib.gemm4_ref(x, lib.unpack_ref(tail, st), "none")
    within(got[:, -200:], ref, err + U[F32] * ref.abs())


# More than 96 rows of e2m1 with a bf16 result go another way (weights widened to bf16).
@pytest.mark.parametrize("M,N,K", [(96, 70, 288), (97, 1, 32), (97, 128, 64), (100, 129, 96), (113, 300, 256), (127, 64, 288), (128, 257, 1056),
                                   (128, 130, 512), (130, 96, 2080), (129, 200, 4128), (256, 40, 1280), (300, 384, 992), (513, 64, 160)])
@pytest.mark.parametrize("epilogue", ["none", "sigmoid"])
def test_gemm4_many_rows(M, N, K, epilogue):
    check_gemm4(M, N, K, "e2m1", 32, None, epilogue, out_dtype=BF16)


def test_gemm4_many_rows_exact():
    """Whole numbers whose products and sums fp32 holds, and a bf16 result too: every code, scale by scale, in its place."""
    M, N, K = 140, 200, 320
    g = gen(3)
    codes = torch.randint(0, 256, (N, K // 2), generator=g, dtype=torch.uint8)
    scales = torch.randint(120, 136, (N, K // 32), generator=g, dtype=torch.uint8)
    x = torch.zeros(M, K)
    at = torch.randint(0, K, (M,), generator=g)
    x[torch.arange(M), at] = 2.0 ** torch.randint(-3, 4, (M,), generator=g)
    got = kda.kda_gemm4(x.to(BF16).cuda(), codes.cuda(), scales.cuda())
    assert torch.equal(f64(got), x.double() @ lib.unpack_ref(codes, scales).T)


@pytest.mark.parametrize("byte", [1, 2, 64, 128, 129, 200, 250, 253])
def test_gemm4_many_rows_scales(byte):
    """Scales from one end to the other, rows of x that bring the results back to where bf16 has them."""
    M, N, K = 99, 65, 256
    g = gen(byte)
    codes, _ = lib.random_weight(g, N, K, fmt="e2m1", group=32)
    scales = torch.full((N, K // 32), byte, dtype=torch.uint8)
    scales[::3] = max(byte - 1, 1)
    x = (randn(g, M, K, dtype=F32) * 2.0 ** min(max(127 - byte, -100), 100)).to(BF16)
    got = kda.kda_gemm4(x.cuda(), codes.cuda(), scales.cuda())
    ref, err = lib.gemm4_ref(x, lib.unpack_ref(codes, scales), "none")
    # what lies below 2^-126 in a product or a sum may be dropped
    within(got, ref, err + U[BF16] * (ref.abs() + err) + K * 2.0 ** -126, f"byte {byte}")


def test_gemm4_many_rows_strides_and_values():
    M, N, K = 130, 140, 416
    g = gen(9)
    x = randn(g, M, K, dtype=BF16)
    codes, scales = lib.random_weight(g, N, K, fmt="e2m1", group=32)
    c, s = codes.cuda(), scales.cuda()
    plain = kda.kda_gemm4(x.cuda(), c, s)
    for offset, pitch in ((0, K + 8), (8, K + 24), (1, K + 8), (0, K + 1), (3, K + 5)):
        big = torch.full((M, pitch + offset), float("nan"), dtype=BF16, device="cuda")
        view = big[:, offset:offset + K]
        view.copy_(x)
        out = torch.full((M + 1, N + 3), 7.0, dtype=BF16, device="cuda")
        kda.kda_gemm4(view, c, s, out=out[:M, 1:N + 1])
        assert torch.equal(out[:M, 1:N + 1], plain)
        assert bool((out[M] == 7).all() and (out[:, 0] == 7).all() and (out[:, N + 1:] == 7).all())
    # a row that is not finite gives what the formula gives and leaves the others alone
    y = x.clone()
    y[5, 17], y[9, 2], y[9, 40], y[66, 0] = float("inf"), float("inf"), float("-inf"), float("nan")
    got = kda.kda_gemm4(y.cuda(), c, s)
    w = lib.unpack_ref(codes, scales)
    keep = [i for i in range(M) if i not in (5, 9, 66)]
    assert torch.equal(got[keep], plain[keep])
    ref = f64(y[[5, 9, 66]]) @ w.T
    have = f64(got[[5, 9, 66]])
    assert torch.equal(torch.isnan(have), torch.isnan(ref)) and torch.equal(torch.isinf(have), torch.isinf(ref))
    assert torch.equal(have[torch.isinf(ref)], ref[torch.isinf(ref)])
    assert torch.equal(kda.kda_gemm4(x.cuda(), c, s), plain)


@pytest.mark.parametrize("M,N,K", [(100, 128, 7168), (128, 256, 7168), (256, 7168, 512), (1000, 140, 2048)])
def test_gemm4_many_rows_split_and_wide(M, N, K):
    check_gemm4(M, N, K, "e2m1", 32, None, out_dtype=BF16)


def close_in_norm(got, ref, units):
    """The error of all outputs together, in units of 2^-24 of theirs: roundings are independent, so those of one kind come to
    one unit at most however many outputs there are, while a systematic loss of bits stands out."""
    err = float((f64(got) - ref).norm() / ref.norm()) * 2.0 ** 24
    assert err <= units, f"{err:.1f} units of 2^-24, {units} allowed"


# A product: roundings of the column (1), of partial sums (each 32 elements' sum and each of the K / 32 additions rounds at
# about the size of the final sum or below, which in norm is sqrt(K / 32) units at most).
@pytest.mark.parametrize("fmt,group,sdt", FORMATS)
@pytest.mark.parametrize("M", [1, 8, 40])
@pytest.mark.parametrize("spread", [False, True])
def test_gemm4_keeps_fp32(M, fmt, group, sdt, spread):
    K = 2048
    g = gen(M + K)
    x = randn(g, M, K, dtype=F32)
    x = (x * randn(g, M, K, dtype=F32) if spread else x).to(BF16)  # products of normal values spread over more exponents
    codes, scales = lib.random_weight(g, 256, K, fmt=fmt, group=group, scale_dtype=sdt)
    got = kda.kda_gemm4(x.cuda(), codes.cuda(), scales.cuda(), out_dtype=F32)
    close_in_norm(got, lib.gemm4_ref(x, lib.unpack_ref(codes, scales), "none")[0], 1 + (K / 32) ** 0.5)


# ------------------------------------------------------------------ mixture of experts
def make_moe(M, E, D, F, fmt, group, sdt, seed, router_dtype=BF16):
    g = gen(seed + M + E + D + F)
    x = randn(g, M, D, dtype=BF16)
    router = randn(g, E, D, std=D ** -0.5, dtype=router_dtype)
    bias = randn(g, E, std=0.05)
    if fmt == "bf16":
        wi, wo = randn(g, E, 2 * F, D, std=D ** -0.5, dtype=BF16), randn(g, E, D, F, std=F ** -0.5, dtype=BF16)
        return x, router, bias, wi, wo, f64(wi), f64(wo)
    wi = lib.random_weight(g, E, 2 * F, D, fmt=fmt, group=group, scale_dtype=sdt)
    wo = lib.random_weight(g, E, D, F, fmt=fmt, group=group, scale_dtype=sdt)
    return x, router, bias, wi, wo, lib.unpack_ref(*wi), lib.unpack_ref(*wo)


def check_moe(M, E, top, D, F, fmt="e2m1", group=32, sdt=None, score="sigmoid", out_dtype=F32, scale=1.0, with_bias=True,
              router_dtype=BF16, x=None, router=None):
    rx, rr, bias, wi, wo, wi64, wo64 = make_moe(M, E, D, F, fmt, group, sdt, 0, router_dtype)
    x, router = rx if x is None else x, rr if router is None else router
    b = bias if with_bias and score == "sigmoid" else None
    pair = lambda w: w.cuda() if isinstance(w, torch.Tensor) else tuple(t.cuda() for t in w)  # noqa: E731
    y, ids, w = kda.kda_moe(x.cuda(), router.cuda(), pair(wi), pair(wo), top, bias=None if b is None else b.cuda(), score=score,
                            scale=scale, out_dtype=out_dtype, return_routing=True)
    ry, rids, rw, bound = lib.moe_ref(x, router, wi64, wo64, top, b, score, scale)
    assert torch.equal(ids.cpu().long(), rids)
    within(w, rw, 2.0 ** -23 * rw.abs(), "weights")
    within(y, ry, bound + U[out_dtype] * (ry.abs() + bound), "y")
    return y


@pytest.mark.parametrize("fmt,group,sdt", FORMATS + [("bf16", 0, None)])
@pytest.mark.parametrize("M,E,top,D,F", [(1, 1, 1, 128, 128), (1, 40, 8, 256, 128), (3, 5, 2, 384, 256), (9, 8, 3, 128, 384),
                                         (20, 4, 4, 256, 128), (33, 300, 5, 128, 128)])
def test_moe_sizes(M, E, top, D, F, fmt, group, sdt):
    check_moe(M, E, top, D, F, fmt, group, sdt)


# Two products in a row, the silu and the product of its two sides (its derivative is at most 1.1: the first products' errors
# pass on about once for the gate and once for the other side, sqrt(2) times), the hidden value's rounding and the weight's,
# the sum over the experts: sqrt(2) (1 + sqrt(D / 32)) + (1 + sqrt(F / 32)) + 4 units.
@pytest.mark.parametrize("fmt,group,sdt", FORMATS + [("bf16", 0, None)])
@pytest.mark.parametrize("M,E,top,D,F", [(1, 6, 3, 1536, 512), (6, 4, 2, 1024, 768), (12, 2, 2, 512, 384)])
def test_moe_keeps_fp32(M, E, top, D, F, fmt, group, sdt):
    x, router, bias, wi, wo, wi64, wo64 = make_moe(M, E, D, F, fmt, group, sdt, 5)
    pair = lambda w: w.cuda() if isinstance(w, torch.Tensor) else tuple(t.cuda() for t in w)  # noqa: E731
    y = kda.kda_moe(x.cuda(), router.cuda(), pair(wi), pair(wo), top, bias=bias.cuda(), out_dtype=F32)
    ref = lib.moe_ref(x, router, wi64, wo64, top, bias, "sigmoid", 1.0)[0]
    close_in_norm(y, ref, 2 ** 0.5 * (1 + (D / 32) ** 0.5) + (1 + (F / 32) ** 0.5) + 4)


@pytest.mark.parametrize("M,E,top,D,F,fmt", [(7, 33, 3, 1056, 352, "int4"), (2, 10, 2, 96, 32, "e2m1"), (5, 6, 2, 72, 40, "bf16"),
                                             (4, 513, 16, 64, 32, "e2m1"), (2, 1024, 32, 64, 64, "int4"), (6, 600, 1, 32, 32, "e2m1")])
def test_moe_odd(M, E, top, D, F, fmt):
    check_moe(M, E, top, D, F, fmt, 32, BF16, scale=2.5)
    check_moe(M, E, top, D, F, fmt, 32, BF16, score="softmax", out_dtype=BF16)


@pytest.mark.parametrize("router_dtype", [BF16, F32])
def test_moe_router_types(router_dtype):
    check_moe(6, 50, 4, 512, 64, router_dtype=router_dtype)
    check_moe(1, 50, 4, 512, 64, router_dtype=router_dtype, with_bias=False)


def test_moe_ties_go_to_the_lower_expert():
    g = gen(2)
    x = randn(g, 5, 64, dtype=BF16)
    router = randn(g, 1, 64, dtype=BF16).expand(12, 64).contiguous()
    rx, _, _, wi, wo, wi64, wo64 = make_moe(5, 12, 64, 32, "e2m1", 32, None, 0)
    _, ids, w = kda.kda_moe(x.cuda(), router.cuda(), tuple(t.cuda() for t in wi), tuple(t.cuda() for t in wo), 5,
                            return_routing=True)
    assert torch.equal(ids.cpu(), torch.arange(5, dtype=torch.int32).expand(5, 5))
    within(w, torch.full((5, 5), 0.2, dtype=torch.float64), 2.0 ** -23 * 0.2)


def test_moe_close_logits_are_told_apart():
    """Logits that differ by less than an fp32 sum of this length can tell."""
    D, E = 4096, 8
    g = gen(4)
    x = randn(g, 3, D, dtype=BF16)
    base = randn(g, D)
    router = base.expand(E, D).contiguous()
    router[:, 7] += torch.linspace(0, 1, E) * 1e-6 * torch.tensor([1.0])
    router = router[torch.randperm(E, generator=g)]
    check_moe(3, E, 3, D, 32, x=x, router=router, router_dtype=F32, with_bias=False)


@pytest.mark.parametrize("with_bias", [True, False])
@pytest.mark.parametrize("low", [-30.0, -85.0, -110.0, -600.0, 90.0])
def test_moe_logits_far_from_zero(low, with_bias):
    """Scores that vanish, or all but reach 1: the weights are their quotients all the same."""
    M, E, D = 3, 9, 64
    x = torch.ones(M, D, dtype=BF16)
    x[1, 0] = 3.0
    router = torch.zeros(E, D)
    router[:, 1] = low - torch.arange(E) * 0.75
    router[:, 0] = torch.linspace(-0.5, 0.5, E)
    check_moe(M, E, 4, D, 32, x=x, router=router, router_dtype=F32, with_bias=with_bias)


@pytest.mark.parametrize("fmt", ["e2m1", "int4", "bf16"])
def test_moe_all_tokens_to_one_expert(fmt):
    """More tokens of an expert than one pass holds columns for."""
    g = gen(6)
    x = randn(g, 70, 256).abs().to(BF16)
    router = randn(g, 64, 256, std=0.01, dtype=BF16)
    router[17] = 0.5
    check_moe(70, 64, 2, 256, 96, fmt, 32, BF16, x=x, router=router, with_bias=False)


@pytest.mark.parametrize("fmt", ["e2m1", "int4", "bf16"])
@pytest.mark.parametrize("M,E,top", [(2, 3, 2), (6, 2, 2), (13, 2, 1), (17, 2, 2), (40, 3, 3), (100, 3, 1)])
def test_moe_many_tokens_per_expert(M, E, top, fmt):
    """Every width of the columns, tokens that fit at once and tokens that do not, several tiles of rows."""
    check_moe(M, E, top, 320, 160, fmt, 32, BF16)


@pytest.mark.parametrize("fmt", ["e2m1", "int4", "bf16"])
def test_moe_long_rows(fmt):
    """More of K than a ring of stages or a segment of columns holds."""
    check_moe(3, 5, 2, 2656, 1312, fmt, 32, F32)


@pytest.mark.parametrize("fmt", ["e2m1", "int4", "bf16"])
def test_moe_not_finite_token(fmt):
    x, router, bias, wi, wo, wi64, wo64 = make_moe(4, 20, 128, 64, fmt, 32, BF16, 1)
    pair = lambda w: w.cuda() if isinstance(w, torch.Tensor) else tuple(t.cuda() for t in w)  # noqa: E731
    call = lambda x: kda.kda_moe(x.cuda(), router.cuda(), pair(wi), pair(wo), 3, bias=bias.cuda(), out_dtype=F32,  # noqa: E731
                                 return_routing=True)
    clean = call(x)
    x[2, 9] = float("nan")
    y, ids, w = call(x)
    assert bool(torch.isnan(y[2]).all()) and bool(torch.isnan(w[2]).all())
    assert torch.equal(ids[2].cpu(), torch.arange(3, dtype=torch.int32))  # NaN ranks last, ties to the lower expert
    keep = [0, 1, 3]
    assert torch.equal(y[keep], clean[0][keep]) and torch.equal(ids[keep], clean[1][keep])


@pytest.mark.parametrize("fmt,group", [("e2m1", 32), ("int4", 64), ("bf16", 0)])
def test_moe_strides_workspace_and_same_bits(fmt, group):
    x, router, bias, wi, wo, _, _ = make_moe(6, 20, 128, 64, fmt, group, F32, 2)
    pair = lambda w: w.cuda() if isinstance(w, torch.Tensor) else tuple(t.cuda() for t in w)  # noqa: E731
    big = torch.zeros(6, 135, dtype=BF16, device="cuda")
    big[:, 3:131] = x.cuda()
    a = kda.kda_moe(x.cuda(), router.cuda(), pair(wi), pair(wo), 4, bias=bias.cuda())
    ybig = torch.full((6, 140), 3.0, dtype=BF16, device="cuda")
    ws = torch.full((1 << 20,), 255, dtype=torch.uint8, device="cuda")
    b = kda.kda_moe(big[:, 3:131], router.cuda(), pair(wi), pair(wo), 4, bias=bias.cuda(), y=ybig[:, 1:129], workspace=ws)
    assert torch.equal(a, b) and bool((ybig[:, 0] == 3).all()) and bool((ybig[:, 129:] == 3).all())
    assert kda.kda_moe(x.cuda()[:0], router.cuda(), pair(wi), pair(wo), 4).shape == (0, 128)


# ------------------------------------------------------------------ verification
def make_verify(lens, V, dtype, seed, agree=0.5, draft=True):
    g = gen(seed + V)
    T = sum(lens)
    logits = torch.randn(T, V, generator=g) * 2
    p = torch.softmax(logits, 1).to(dtype)
    q = torch.softmax(logits + agree * torch.randn(T, V, generator=g), 1).to(dtype) if draft else None
    src = q.float() if draft else p.float()
    tokens = (src / -torch.log(torch.rand(T, V, generator=g).clamp(min=1e-30))).argmax(1) if T else torch.zeros(0)
    u = torch.rand(T, generator=g)
    cu = np.zeros(len(lens) + 1, np.int32)
    cu[1:] = np.cumsum(lens)
    return p, q, tokens.int(), u, cu


def check_verify(p, q, tokens, u, cu, **kw):
    out, acc = kda.kda_verify(p.cuda(), tokens.cuda(), u.cuda(), cu, draft=None if q is None else q.cuda(), **kw)
    ro, ra = lib.verify_ref(p, q, tokens, u, cu)
    assert out.dtype == tokens.dtype
    assert np.array_equal(acc.cpu().numpy(), ra)
    assert np.array_equal(out.cpu().numpy(), ro)
    return out, acc


@pytest.mark.parametrize("lens", [[1], [8], [4, 4, 4], [0, 3, 1, 0, 8, 2, 0], [2] * 40, [5] * 400])
@pytest.mark.parametrize("V", [1, 7, 100, 2047, 2049, 4101])
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("draft", [True, False])
def test_verify_sizes(lens, V, dtype, draft):
    check_verify(*make_verify(lens, V, dtype, len(lens), draft=draft))


@pytest.mark.parametrize("V", [32003, 160000, 300001])
@pytest.mark.parametrize("agree", [0.05, 1.5])
def test_verify_large_vocabularies(V, agree):
    for lens in ([3], [4, 2, 5], [2, 1] * 40):
        if sum(lens) * V <= 1 << 24:
            check_verify(*make_verify(lens, V, F32, len(lens), agree))


def test_verify_thresholds():
    """u of 0, u next to 1, and shares of nothing around every step."""
    V, n = 5000, 64
    p = torch.zeros(n, V)
    g = gen(9)
    for i in range(n):
        at = torch.randperm(V, generator=g)[:1 + i % 5]
        p[i, at] = torch.rand(len(at), generator=g) + 0.1
    u = torch.tensor([0.0, 1.0 - 2.0 ** -24, 0.5, 0.25])[torch.arange(n) % 4]
    check_verify(p, None, torch.zeros(n, dtype=torch.int32), u, np.arange(n + 1, dtype=np.int32))


def test_verify_rows_with_nothing():
    """Equal distributions leave no residual, a row of zeros leaves nothing at all."""
    V = 3000
    p, q, tokens, u, cu = make_verify([3, 3, 3, 2], V, F32, 1)
    q[0] = p[0] * 2  # below the drafter everywhere
    u[0] = 0.9
    p[3] = 0
    p[6, :] = 0
    q[6, :] = 0
    p[7] = float("nan")
    p[9] = -1
    tokens[1] = V + 5  # outside: never taken
    tokens[4] = -3
    out, acc = check_verify(p, q, tokens, u, cu)
    assert int(out[6]) == -1 and int(acc[2]) == 0
    check_verify(p, None, tokens.long(), u, cu)


def test_verify_strides_tails_and_device_cu():
    V = 1001
    p, q, tokens, u, cu = make_verify([2, 4, 1], V, BF16, 3)
    ro, ra = lib.verify_ref(p, q, tokens, u, cu)
    bp, bq = torch.zeros(7, 1100, dtype=BF16, device="cuda"), torch.zeros(7, 1207, dtype=BF16, device="cuda")
    bp[:, 5:5 + V], bq[:, 2:2 + V] = p.cuda(), q.cuda()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out, acc = kda.kda_verify(bp[:, 5:5 + V], tokens.cuda(), u.cuda(), cu, draft=bq[:, 2:2 + V], d_status=status,
                              check_cu_on_host=False)
    assert np.array_equal(out.cpu().numpy(), ro) and np.array_equal(acc.cpu().numpy(), ra) and int(status) == 0


def test_verify_offsets_past_32_bits():
    """Rows of both distributions that lie more than 2^32 bytes apart."""
    V, far = 1003, 1200000001
    if torch.cuda.mem_get_info()[0] < 16 << 30:
        pytest.skip("needs 16 GB of free memory")
    p, q, tokens, u, cu = make_verify([3, 1], V, BF16, 4)
    held = [torch.empty(3 * far + V, dtype=BF16, device="cuda") for _ in range(2)]
    wide = [h.as_strided((4, V), (far, 1)) for h in held]
    wide[0].copy_(p), wide[1].copy_(q)
    out, acc = kda.kda_verify(wide[0], tokens.cuda(), u.cuda(), cu, draft=wide[1])
    ro, ra = lib.verify_ref(p, q, tokens, u, cu)
    assert np.array_equal(out.cpu().numpy(), ro) and np.array_equal(acc.cpu().numpy(), ra)


def test_verify_expected_share():
    """Over evenly spread u the accepted drafts and the drawn tokens have the target's distribution."""
    V, n = 6, 20000
    g = gen(8)
    p = torch.tensor([0.05, 0.3, 0.1, 0.25, 0.2, 0.1])
    q = torch.tensor([0.3, 0.1, 0.2, 0.1, 0.1, 0.2])
    tokens = torch.multinomial(q, 2 * n, replacement=True, generator=g).int()
    u = torch.rand(2 * n, generator=g)
    cu = np.arange(0, 2 * n + 1, 2, dtype=np.int32)
    out, _ = check_verify(p.expand(2 * n, V).contiguous(), q.expand(2 * n, V).contiguous(), tokens, u, cu)
    first = out.view(n, 2)[:, 0].cpu().long()
    share = torch.bincount(first, minlength=V).double() / n
    # six standard deviations of a share of n draws
    assert bool(((share - p.double()).abs() < 6 * (p.double() * (1 - p.double()) / n).sqrt()).all())


# ------------------------------------------------------------------ together, streams, captures
def test_one_speculative_step():
    """Projection, experts, vocabulary rows and verification as a decode step runs them, against the same chain in 64
    bits from each operator's own inputs."""
    M, D, V = 12, 256, 1000
    g = gen(20)
    x = randn(g, M, D, dtype=BF16).cuda()
    wp = kda.kda_pack4(randn(g, D, D, std=D ** -0.5).cuda())
    head = kda.kda_pack4(randn(g, V, D, std=0.2).cuda(), format="int4", group=128)
    _, router, bias, wi, wo, wi64, wo64 = make_moe(M, 16, D, 128, "e2m1", 32, None, 5)
    cu = np.array([0, 4, 8, 12], np.int32)
    u = torch.rand(M, generator=g)

    def step():
        h = kda.kda_gemm4(x, *wp)
        y = kda.kda_moe(h, router.cuda(), tuple(t.cuda() for t in wi), tuple(t.cuda() for t in wo), 4, bias=bias.cuda())
        logits = kda.kda_gemm4(y, *head, out_dtype=F32)
        p = torch.softmax(logits, 1)
        tokens = p.argmax(1).int()
        return h, y, logits, p, tokens, *kda.kda_verify(p, tokens, u.cuda(), cu)

    h, y, logits, p, tokens, out, acc = step()
    ref, err = lib.gemm4_ref(x, lib.unpack_ref(*wp), "none")
    within(h, ref, err + U[BF16] * (ref.abs() + err))
    ry, _, _, bound = lib.moe_ref(h, router, wi64, wo64, 4, bias, "sigmoid", 1.0)
    within(y, ry, bound + U[BF16] * (ry.abs() + bound))
    ref, err = lib.gemm4_ref(y, lib.unpack_ref(*head), "none")
    within(logits, ref, err + U[F32] * (ref.abs() + err))
    ro, ra = lib.verify_ref(p.cpu(), None, tokens.cpu(), u, cu)
    assert np.array_equal(out.cpu().numpy(), ro) and np.array_equal(acc.cpu().numpy(), ra)


@pytest.mark.parametrize("fmt", ["e2m1", "int4", "bf16"])
def test_streams_and_captures(fmt):
    """The same bits on another stream and from a replayed graph with new inputs."""
    x, router, bias, wi, wo, _, _ = make_moe(5, 24, 256, 128, fmt, 32, BF16, 7)
    x, router, bias = dev(x, router, bias)
    wi, wo = (w.cuda() if isinstance(w, torch.Tensor) else tuple(t.cuda() for t in w) for w in (wi, wo))
    e2m1 = tuple(t.cuda() for t in lib.random_weight(gen(2), 300, 256, fmt="e2m1", group=32))
    codes, scales = (t.cuda() for t in lib.random_weight(gen(1), 300, 256, fmt="int4", group=64, scale_dtype=F32))
    p, q, tokens, u, cu = make_verify([4, 3, 5], 5000, F32, 2)
    p, q, tokens, u = dev(p, q, tokens, u)
    pair = (torch.from_numpy(cu).cuda(), cu)

    def run(stream=None):
        y, ids, w = kda.kda_moe(x, router, wi, wo, 4, bias=bias, return_routing=True, stream=stream)
        return [y, ids, w, kda.kda_gemm4(x, codes, scales, stream=stream), kda.kda_gemm4(x, *e2m1, stream=stream),
                *kda.kda_verify(p, tokens, u, pair, draft=q, stream=stream), *kda.kda_pack4(x, stream=stream)]

    want = run()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = run(s)
    torch.cuda.current_stream().wait_stream(s)
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = run()
    x.copy_(x.flip(0))
    u.copy_(1 - u)
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(run(), held))


def test_calls_side_by_side():
    """Calls on several streams at once, each with its own workspace, give the bits of calls one after another."""
    sets = []
    for i, fmt in enumerate(("e2m1", "int4", "bf16", "e2m1")):
        x, router, bias, wi, wo, _, _ = make_moe(9, 40, 512, 256, fmt, 32, BF16, 30 + i)
        w = [v.cuda() if isinstance(v, torch.Tensor) else tuple(t.cuda() for t in v) for v in (wi, wo)]
        sets.append((*dev(x, router, bias), *w, tuple(t.cuda() for t in lib.random_weight(gen(i), 700, 512, fmt="e2m1", group=32))))

    def call(x, router, bias, wi, wo, w4, stream=None):
        return [kda.kda_moe(x, router, wi, wo, 5, bias=bias, stream=stream), kda.kda_gemm4(x, *w4, stream=stream)]

    want = [call(*s) for s in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    for _ in range(5):
        got = [call(*s, stream=st) for s, st in zip(sets, streams)]
        torch.cuda.synchronize()
        for a, b in zip(want, got):
            assert all(torch.equal(p, q) for p, q in zip(a, b))


@pytest.mark.parametrize("M", [130, 300])
def test_many_rows_in_a_chain(M):
    """Products whose rows another product wrote just before, beside other calls on other streams, and replayed."""
    K, N = 1024, 640
    g = gen(M)
    x = randn(g, M, K, dtype=BF16).cuda()
    w1 = tuple(t.cuda() for t in lib.random_weight(g, N, K, fmt="e2m1", group=32))
    w2 = tuple(t.cuda() for t in lib.random_weight(g, K, N, fmt="e2m1", group=32))

    def chain(x, stream=None):
        for _ in range(4):
            x = kda.kda_gemm4(kda.kda_gemm4(x, *w1, stream=stream), *w2, stream=stream)
        return x

    want, few = chain(x), chain(x[:20])
    torch.cuda.synchronize()
    assert torch.isfinite(want).all()
    streams = [torch.cuda.Stream() for _ in range(4)]
    for _ in range(5):
        got = [chain(x if i % 2 else x[:20], s) for i, s in enumerate(streams)]
        torch.cuda.synchronize()
        assert all(torch.equal(y, want if i % 2 else few) for i, y in enumerate(got))
    held_in = x.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = chain(held_in)
    held_in.copy_(x.flip(0))
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(held, chain(x.flip(0))) and torch.equal(held, want.flip(0))


def test_after_the_multi_token_decode():
    """A step as it is run: the layer decodes each sequence's last token and its drafts from kept states, projections in 4 bits
    on both sides, the drafts are verified, and the layer runs again over what was accepted."""
    H, D, N, V = 2, 128, 3, 600
    width = H * D
    g = gen(40)
    lens = [4, 2, 5]
    cu = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
    T = int(cu[-1])
    x = randn(g, T, width, dtype=BF16).cuda()
    proj = [kda.kda_pack4(randn(g, width, width, std=width ** -0.5).cuda()) for _ in range(3)]
    gates = kda.kda_pack4(randn(g, width, width, std=width ** -0.5).cuda(), format="int4", group=64, scale_dtype=F32)
    head = kda.kda_pack4(randn(g, V, width, std=3 * width ** -0.5).cuda())
    conv_w = randn(g, 3, width, 4, std=0.5).cuda()
    beta = torch.rand(T, H, generator=g).cuda()
    state, conv = torch.randn(N, H, D, D, generator=g).cuda() * 0.02, randn(g, N, 3 * width, 3, dtype=BF16).cuda()
    router, wi, wo = (randn(g, *s, std=0.06, dtype=BF16).cuda() for s in ((8, width), (8, 256, width), (8, width, 128)))

    def layer(rows, cu):
        t = rows.shape[0]
        q, k, v = (kda.kda_gemm4(rows, *w).view(t, H, D) for w in proj)
        decay = kda.kda_gemm4(rows, *gates, epilogue="decay").view(t, H, D)
        b = beta[:t].contiguous()
        out, fin = kda.kda_prefill(q, k, v, conv_w, decay, b, cu, initial_state=state, conv_state_in=conv,
                                   conv_state_out=torch.empty_like(conv))
        y = kda.kda_moe(out.reshape(t, width), router, wi, wo, 2, score="softmax")
        return torch.softmax(kda.kda_gemm4(y, *head, out_dtype=F32), 1), fin

    probs, _ = layer(x, cu)
    drafts = probs.argmax(1)
    drafts[2] = (drafts[2] + 1) % V  # not the target's best
    u = torch.full((T,), 0.3).cuda()
    tokens, accepted = kda.kda_verify(probs, drafts, u, cu)
    ro, ra = lib.verify_ref(probs.cpu(), None, drafts.cpu(), u.cpu(), cu)
    assert np.array_equal(tokens.cpu().numpy(), ro) and np.array_equal(accepted.cpu().numpy(), ra)
    # the states of what stands: the sequences again, as far as they were accepted
    keep = accepted.cpu().numpy() + 1
    rows = torch.cat([x[cu[i]:cu[i] + keep[i]] for i in range(N)])
    again, fin = layer(rows, np.concatenate([[0], np.cumsum(keep)]).astype(np.int32))
    assert fin.shape == state.shape and bool(torch.isfinite(fin).all()) and again.shape == (int(keep.sum()), V)
