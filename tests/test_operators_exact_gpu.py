"""The products on whole numbers, whose sums are exact in 32 bits in any order:
every kernel, tile and split has to give the exact result, so a lost or doubled
step of a long contraction shows as a wrong number.  Each case names the tile
and the split that it is there for."""
import pytest
import torch

import compiler_hlo_amd as H

pytestmark = pytest.mark.gpu

T = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16, "s8": torch.int8,
     "f8e4m3": torch.float8_e4m3fn}


def whole(g, shape, dtype, top=2):
    """Whole numbers -top .. top: exact in every operand type, as are their
    products; 16384 products of 4 at most stay below 2^24."""
    return torch.randint(-top, top + 1, shape, generator=g, device="cuda").to(torch.float32).to(T[dtype])


def powers(g, n):
    """Scales that round nothing."""
    return torch.exp2(torch.randint(-3, 2, (n,), generator=g, device="cuda").float())


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def same(got, want, dtype, slack=None):
    """`want` (64 bits, exact) rounded once to dtype.  slack: e4m3's matrix
    instructions may err by 2^-17 of the sum of magnitudes before that."""
    rounded = want.to(torch.float32).to(T[dtype])
    if slack is None:
        bad = (got != rounded)
    else:
        half = torch.finfo(T[dtype]).eps / 2
        bad = ~((got.double() - want).abs() <= slack + want.abs() * half * (1 + 2.0 ** -7))
    assert not bad.any(), "%d of %d differ; first at %s: got %r, want %r" % (
        int(bad.sum()), bad.numel(), bad.nonzero()[0].tolist(), float(got[bad][0]), float(rounded[bad][0]))


def magnitude(a, b):
    return a.double().abs() @ b.double().abs().t()


# rows, columns and splits of a tile; 0 splits: more than one
BIG, SMALL, STRIP, SKINNY = (256, 256), (128, 128), (64, 128), (16, 16)
PRODUCTS = [
    # the larger tile: two and three stages, ragged edges and contractions
    ("bf16", 4096, 4096, 136, BIG, 1), ("f16", 4096, 4096, 192, BIG, 1), ("s8", 4096, 4096, 272, BIG, 1),
    ("f8e4m3", 4096, 4096, 400, BIG, 1), ("f16", 4081, 4090, 250, BIG, 1), ("s8", 4081, 4090, 250, BIG, 1),
    # whole tiles, then tiles shared by several workgroups
    ("bf16", 4400, 4100, 2200, BIG, 0), ("f16", 4400, 4100, 2112, BIG, 0), ("s8", 4400, 4100, 4096, BIG, 0),
    ("f8e4m3", 4400, 4100, 4096, BIG, 0), ("bf16", 4224, 4096, 1000, BIG, 0),
    # the smaller tile, whole and shared, an odd and an even number of stages
    ("bf16", 2305, 8200, 520, SMALL, 1), ("f16", 300, 2000, 16384, SMALL, 0), ("s8", 700, 1000, 8192, SMALL, 0),
    ("f8e4m3", 700, 1000, 8192, SMALL, 0), ("bf16", 1100, 1030, 8200, SMALL, 0), ("f16", 65, 100, 4160, SMALL, 0),
    # strips, whole and shared
    ("bf16", 64, 4096, 4096, STRIP, 0), ("f16", 33, 4100, 8200, STRIP, 0), ("s8", 17, 1000, 16384, STRIP, 0),
    ("f8e4m3", 9, 520, 16384, STRIP, 0), ("bf16", 64, 33000, 1000, STRIP, 1), ("s8", 8, 8400, 4000, STRIP, 1),
    # a few rows: 16 waves a workgroup, 8 of them, and shared by several workgroups
    ("bf16", 1, 4096, 16384, SKINNY, 1), ("f16", 8, 4096, 4200, SKINNY, 1), ("s8", 5, 5000, 8200, SKINNY, 1),
    ("f8e4m3", 8, 5120, 4096, SKINNY, 1),
    ("bf16", 1, 5200, 4096, SKINNY, 1), ("f16", 5, 8192, 2056, SKINNY, 1), ("s8", 8, 6001, 4096, SKINNY, 1),
    ("f8e4m3", 8, 8192, 5000, SKINNY, 1), ("bf16", 8, 6000, 8200, SKINNY, 1),
    ("bf16", 2, 24, 16384, SKINNY, 0), ("f16", 8, 512, 16000, SKINNY, 0), ("s8", 1, 100, 16384, SKINNY, 0),
    ("f8e4m3", 3, 300, 16384, SKINNY, 0),
]


@pytest.mark.parametrize("dtype, m, n, k, tile, splits", PRODUCTS)
def test_matmul(dtype, m, n, k, tile, splits):
    g = gen(m + n + k)
    a, b = whole(g, (m, k), dtype), whole(g, (n, k), dtype)
    z = a.double() @ b.double().t()
    slack = magnitude(a, b) * 2.0 ** -17 if dtype == "f8e4m3" else None
    params = [a, b]
    if dtype in ("s8", "f8e4m3"):
        sa, sb = powers(g, m), powers(g, n)
        params += [sa, sb]
        scale = sa.double()[:, None] * sb.double()
        z, slack = z * scale, None if slack is None else slack * scale
    # results in 16 bits where 8-bit sums in 32 bits take another kernel
    for out in ("bf16", "f16") if dtype == "f8e4m3" else ("f32", "bf16"):
        op = H.Matmul(m, n, k, dtype, out_dtype=out)
        plan = op.plan()
        assert (plan["tile_rows"], plan["tile_cols"]) == tile and (plan["splits"] == 1) == (splits == 1), plan
        print("matmul", dtype, out, m, n, k, plan, flush=True)
        same(op(*params), z, out, slack)
    if dtype != "f8e4m3":
        bias, residual = whole(g, (n,), "f32"), whole(g, (m, n), "f32")
        op = H.Matmul(m, n, k, dtype, out_dtype="f32", bias=True, activation="relu", residual=True, save=True)
        d, saved = op(*params, bias, residual)
        same(saved, z + bias.double(), "f32")
        same(d, (z + bias.double()).clamp(min=0) + residual.double(), "f32")


@pytest.mark.parametrize("m, n, k", [(1, 4096, 4096), (8, 300, 16384), (3, 6000, 2000), (40, 2000, 4096),
                                     (300, 520, 8192), (2000, 2100, 400)])
def test_matmul_f8_to_f32(m, n, k):
    """e4m3 widened to 16 bits: sums to f32's rounding, here exact."""
    g = gen(m + k)
    a, b, sa, sb = whole(g, (m, k), "f8e4m3"), whole(g, (n, k), "f8e4m3"), powers(g, m), powers(g, n)
    z = (a.double() @ b.double().t()) * (sa.double()[:, None] * sb.double())
    same(H.Matmul(m, n, k, "f8e4m3", out_dtype="f32")(a, b, sa, sb), z, "f32")
    if n % 2 == 0:
        d, saved = H.GatedFeedForward(m, n // 2, k, "f8e4m3", out_dtype="f32", activation="relu", save=True)(a, b, sa, sb)
        same(saved, z, "f32")
        f, u = z[:, :n // 2].clamp(min=0), z[:, n // 2:]
        same(d, f * u, "f32", (f * u).abs() * 2.0 ** -24)


GATED = [
    ("bf16", 4096, 2048, 136, BIG, 1), ("f16", 4081, 2047, 250, BIG, 1), ("s8", 2100, 2200, 2048, BIG, 1),
    ("f8e4m3", 2100, 2200, 2048, BIG, 1),
    ("bf16", 700, 11264, 1024, BIG, 0), ("f16", 700, 11264, 2120, BIG, 0), ("s8", 700, 11264, 4096, BIG, 0),
    ("f8e4m3", 700, 11264, 4096, BIG, 0),
    ("bf16", 1000, 4500, 2048, SMALL, 0), ("s8", 2200, 4200, 256, SMALL, 1), ("f16", 2200, 4201, 456, SMALL, 1),
    ("bf16", 24, 11264, 1000, STRIP, 1), ("s8", 40, 1000, 8192, STRIP, 0), ("f16", 9, 520, 4096, STRIP, 0),
    ("bf16", 1, 2048, 4096, (16, 32), 1), ("f16", 8, 4096, 2056, (16, 32), 1), ("s8", 5, 100, 16384, (16, 32), 0),
    ("f8e4m3", 8, 1000, 16384, (16, 32), 0),
]


@pytest.mark.parametrize("dtype, m, n, k, tile, splits", GATED)
def test_gated(dtype, m, n, k, tile, splits):
    g = gen(m + n + k)
    a, b = whole(g, (m, k), dtype), whole(g, (2 * n, k), dtype)
    z = a.double() @ b.double().t()
    slack = magnitude(a, b) * 2.0 ** -17 if dtype == "f8e4m3" else None
    params = [a, b]
    if dtype in ("s8", "f8e4m3"):
        sa, sb = powers(g, m), powers(g, 2 * n)
        params += [sa, sb]
        scale = sa.double()[:, None] * sb.double()
        z, slack = z * scale, None if slack is None else slack * scale
    f, u = z[:, :n].clamp(min=0), z[:, n:]
    out = "bf16" if dtype == "f8e4m3" else "f32"
    op = H.GatedFeedForward(m, n, k, dtype, out_dtype=out, activation="relu", save=True)
    plan = op.plan()
    assert (plan["tile_rows"], plan["tile_cols"]) == tile and (plan["splits"] == 1) == (splits == 1), plan
    print("gated", dtype, m, n, k, plan, flush=True)
    d, saved = op(*params)
    same(saved, z, out, slack)
    # f u is one rounding in 32 bits, and then the result's own
    e = (f * u).abs() * 2.0 ** -24
    if slack is not None:
        e = e + slack[:, :n] * (u.abs() + slack[:, n:]) + f * slack[:, n:]
    same(d, f * u, out, e)


# one launch makes both products; "shared" of at least one of them
GRADS = [("bf16", 4096, 4096, 192, SMALL), ("f16", 4096, 4096, 4096, BIG), ("bf16", 4096, 8192, 2048, BIG),
         ("f16", 4200, 4100, 4100, BIG), ("bf16", 4100, 4352, 1024, BIG), ("f16", 2100, 9000, 2100, BIG),
         ("bf16", 2304, 4400, 4100, BIG), ("bf16", 1100, 17000, 1030, SMALL), ("f16", 589, 832, 640, SMALL),
         ("f16", 2304, 2200, 2120, SMALL), ("bf16", 100, 100, 8200, SMALL), ("bf16", 8200, 70, 130, SMALL)]


@pytest.mark.parametrize("dtype, m, n, k, tile", GRADS)
def test_matmul_grad(dtype, m, n, k, tile):
    g = gen(m + n + k)
    dd, a, b, z = whole(g, (m, n), dtype), whole(g, (m, k), dtype), whole(g, (n, k), dtype), whole(g, (m, n), dtype)
    for act, bias in ((None, True), ("relu", True), (None, False)):
        op = H.MatmulGrad(m, n, k, dtype, bias=bias, activation=act)
        plan = op.plan()
        assert (plan["tile_rows"], plan["tile_cols"]) == tile, plan
        print("matmul_grad", dtype, m, n, k, act, plan, flush=True)
        dz = dd.double() * (z > 0) if act else dd.double()
        got = op(*([dd, a, b] + ([z] if act else [])))
        same(got[0], dz @ b.double(), dtype)
        same(got[1], dz.t() @ a.double(), dtype)
        if bias:
            same(got[2], dz.sum(0), "f32")


@pytest.mark.parametrize("dtype, m, n, k, tile", [
    ("bf16", 2100, 2200, 2048, BIG), ("f16", 1030, 4500, 4100, BIG), ("bf16", 2100, 4400, 2050, BIG),
    ("f16", 4096, 2048, 256, SMALL), ("bf16", 4100, 2201, 1030, BIG), ("bf16", 200, 1030, 520, SMALL),
    ("f16", 1000, 129, 1000, SMALL)])
def test_gated_grad(dtype, m, n, k, tile):
    g = gen(m + n + k)
    dd, a, b, z = whole(g, (m, n), dtype, 1), whole(g, (m, k), dtype), whole(g, (2 * n, k), dtype), whole(g, (m, 2 * n), dtype)
    op = H.GatedFeedForwardGrad(m, n, k, dtype, activation="relu")
    plan = op.plan()
    assert (plan["tile_rows"], plan["tile_cols"]) == tile, plan
    print("gated_grad", dtype, m, n, k, plan, flush=True)
    gate, up = z[:, :n].double(), z[:, n:].double()
    dz = torch.cat([dd.double() * up * (gate > 0), dd.double() * gate.clamp(min=0)], 1)
    da, db = op(dd, a, b, z)
    same(da, dz @ b.double(), dtype)
    same(db, dz.t() @ a.double(), dtype)


@pytest.mark.parametrize("dtype, m, n, k", [
    ("bf16", 4099, 4096, 4096), ("f16", 4160, 4096, 4096), ("s8", 4099, 4096, 16384), ("f8e4m3", 4110, 4096, 16384)])
def test_last_rows(dtype, m, n, k):
    """A few rows past whole tiles as a product of their own: 256 tiles in one
    round, then a skinny product or a strip; every operand and result of theirs
    lies at an offset, rows further apart than their length."""
    g = gen(m + k)
    a, b = whole(g, (m, k), dtype), whole(g, (n, k), dtype)
    z = a.double() @ b.double().t()
    slack = magnitude(a, b) * 2.0 ** -17 if dtype == "f8e4m3" else None
    params = [a, b]
    if dtype in ("s8", "f8e4m3"):
        sa, sb = powers(g, m), powers(g, n)
        params += [sa, sb]
        scale = sa.double()[:, None] * sb.double()
        z, slack = z * scale, None if slack is None else slack * scale
    out = "bf16" if dtype == "f8e4m3" else "f32"
    bias = whole(g, (n,), out)
    residual = torch.zeros((m, n + 24), dtype=T[out], device="cuda")[:, 8:n + 8]
    residual.copy_(whole(g, (m, n), out))
    op = H.Matmul(m, n, k, dtype, out_dtype=out, bias=True, activation="relu", residual=True, save=True,
                  strides={"residual": n + 24, "d": n + 8, "z": n + 16})
    plan = op.plan()
    assert (plan["tile_rows"], plan["splits"]) == (256, 1) and -(-m // 256) * -(-n // 256) > 256, plan
    d, saved = op(*params, bias, residual)
    same(saved, z + bias.double(), out, slack)
    same(d, (z + bias.double()).clamp(min=0) + residual.double(), out, slack)


@pytest.mark.parametrize("dtype, m, n, k", [("bf16", 4099, 2048, 8192), ("f8e4m3", 4110, 2048, 4096), ("s8", 2060, 4096, 4096)])
def test_gated_last_rows(dtype, m, n, k):
    g = gen(m + k)
    a, b = whole(g, (m, k), dtype), whole(g, (2 * n, k), dtype)
    z = a.double() @ b.double().t()
    slack = magnitude(a, b) * 2.0 ** -17 if dtype == "f8e4m3" else torch.zeros_like(z)
    params = [a, b]
    if dtype != "bf16":
        sa, sb = powers(g, m), powers(g, 2 * n)
        params += [sa, sb]
        scale = sa.double()[:, None] * sb.double()
        z, slack = z * scale, slack * scale
    out = "bf16" if dtype == "f8e4m3" else "f32"
    op = H.GatedFeedForward(m, n, k, dtype, out_dtype=out, activation="relu", save=True,
                            strides={"d": n + 8, "z": 2 * n + 8})
    plan = op.plan()
    assert (plan["tile_rows"], plan["splits"]) == (256, 1) and -(-m // 256) * -(-n // 128) > 256, plan
    d, saved = op(*params)
    same(saved, z, out, slack)
    f, u = z[:, :n].clamp(min=0), z[:, n:]
    same(d, f * u, out, (f * u).abs() * 2.0 ** -24 + slack[:, :n] * (u.abs() + slack[:, n:]) + f * slack[:, n:])
