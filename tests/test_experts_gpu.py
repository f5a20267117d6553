"""The operators by expert and with block scales on the GPU against plain
64-bit forms: types, directions, sizes at which a kernel or tile changes, odd
lengths, strides, experts without rows, rows that are no expert's, streams and
graphs."""
import pytest
import torch

import compiler_hlo_amd as H
import experts_reference as X
import operators_reference as R
from test_operators_gpu import T, eight, gen, normal, say

pytestmark = pytest.mark.gpu


def same(got, want):
    for g, w in zip(got, want):
        assert torch.equal(g.cpu(), w), (g, w)


# --------------------------------------------------------------------------
# sort
# --------------------------------------------------------------------------
# one workgroup up to 8192 pairs, chunks beyond; runs that end inside 64 pairs
SORTS = [(1, 1, 1), (1, 8, 64), (3, 2, 5), (24, 8, 128), (65, 7, 33), (64, 16, 1024), (1024, 8, 64), (1025, 8, 64),
         (9001, 7, 100), (20000, 1, 2), (65536, 8, 256), (70001, 3, 1000), (0, 2, 5)]


@pytest.mark.parametrize("tokens, top_k, experts", SORTS)
def test_sort(tokens, top_k, experts):
    g = gen(tokens + 31 * experts)
    ids = torch.randint(0, experts, (tokens, top_k), generator=g, dtype=torch.int32)
    wild = torch.randint(-2 ** 31, 2 ** 31 - 1, (tokens, top_k), generator=g).to(torch.int32)
    near = torch.randint(-experts, 2 * experts, (tokens, top_k), generator=g, dtype=torch.int32)
    for name, v in (("all", ids), ("some", near), ("wild", wild), ("one", ids * 0 + experts - 1), ("none", ids * 0 - 1)):
        say("sort", tokens, top_k, experts, name)
        got = H.ExpertSort(tokens, top_k, experts)(v.cuda())
        same(got, X.sort(v, experts))


def test_sort_strides():
    g = gen(4)
    for tokens, top_k, experts in ((37, 3, 9), (5000, 4, 300)):
        full = torch.randint(0, experts, (tokens, top_k + 5), generator=g, dtype=torch.int32).cuda()
        op = H.ExpertSort(tokens, top_k, experts, strides={"expert": top_k + 5, "place": top_k + 2})
        got = op(full[:, :top_k])
        assert got[0].stride(0) == top_k + 2
        same(got, X.sort(full[:, :top_k].contiguous(), experts))


# --------------------------------------------------------------------------
# dispatch, combine
# --------------------------------------------------------------------------
def chosen(g, tokens, top_k, experts, shard):
    """(ids, place, order, offsets); in a shard some pairs have no row."""
    lo, hi = (-(experts // 2) - 1, experts + experts // 2 + 1) if shard else (0, experts)
    ids = torch.randint(lo, hi, (tokens, top_k), generator=g, dtype=torch.int32)
    return [ids] + X.sort(ids, experts)


LAYOUTS = [(1, 8, 64, 4096), (3, 2, 5, 7), (24, 8, 128, 1000), (129, 1, 3, 64), (300, 5, 16, 2056), (65, 11, 40, 4104),
           (2, 20, 30, 513), (500, 3, 7, 16391), (33, 2, 4, 1), (1000, 9, 20, 130),
           (700, 2, 8, 1024), (515, 4, 9, 65)]


@pytest.mark.parametrize("tokens, top_k, experts, cols", LAYOUTS)
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32", "s8", "f8e4m3"])
def test_dispatch(dtype, tokens, top_k, experts, cols):
    for shard in (False, True):
        say("dispatch", dtype, tokens, top_k, experts, cols, shard)
        g = gen(tokens + cols)
        _, place, order, _ = chosen(g, tokens, top_k, experts, shard)
        count = int((order >= 0).sum())
        token = order[:count] // top_k
        for stride in (None, cols + 3):
            strides = {} if stride is None else {"x": stride, "y": stride + 2, "place": top_k + 1}
            p = torch.zeros((tokens, top_k + (0 if stride is None else 1)), dtype=torch.int32, device="cuda")[:, :top_k]
            p.copy_(place)
            for scales in ([None, "blocks"] if dtype == "f8e4m3" else [None]):
                op = H.ExpertDispatch(tokens, top_k, cols, dtype, scales=scales, strides=strides)
                if dtype in ("s8", "f8e4m3"):
                    x, _ = eight(g, tokens, cols, dtype)
                    s = torch.rand((-(-cols // 128), tokens) if scales else (tokens,), generator=g).cuda()
                    if stride is not None:
                        wide = torch.zeros((tokens, stride), dtype=T[dtype], device="cuda")
                        wide[:, :cols] = x
                        x = wide[:, :cols]
                    params = [x, p, s]
                else:
                    x = normal(g, (tokens, cols), dtype, stride=stride)
                    params = [x, p]
                out = [b.empty("cuda") for b in op.results]
                bits = {1: torch.int8, 2: torch.int16, 4: torch.int32}
                before = []
                for t in out:
                    t.view(bits[t.element_size()]).fill_(85)
                    before.append(t.clone())
                got = op(*params, out=out)
                got = [got] if isinstance(got, torch.Tensor) else list(got)
                as_bits = lambda t: t.contiguous().view(bits[t.element_size()]).cpu()  # noqa: E731
                assert torch.equal(as_bits(got[0][:count]), as_bits(x)[token])
                assert torch.equal(as_bits(got[0][count:]), as_bits(before[0][count:])), "rows of no expert changed"
                if len(got) > 1:
                    want = s.cpu()[:, token] if scales else s.cpu()[token]
                    assert torch.equal(got[1].cpu()[..., :count], want)
                    assert torch.equal(as_bits(got[1][..., count:]), as_bits(before[1][..., count:]))


def rows_at(y, place):
    """[tokens, top_k, cols] in 64 bits, zeros where there is no row."""
    rows = R.f64(y)[place.clamp(min=0).long()]
    return torch.where((place >= 0)[:, :, None], rows, 0.0)


@pytest.mark.parametrize("tokens, top_k, experts, cols", LAYOUTS)
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
def test_combine(dtype, tokens, top_k, experts, cols):
    for i, (shard, weighted, res, stride) in enumerate([(False, True, False, None), (True, True, True, cols + 5),
                                                        (True, False, True, None), (False, False, False, cols + 8)]):
        say("combine", dtype, tokens, top_k, experts, cols, shard, weighted, res, stride)
        g = gen(tokens + cols + i)
        _, place, order, _ = chosen(g, tokens, top_k, experts, shard)
        pairs, count = tokens * top_k, int((order >= 0).sum())
        y = normal(g, (pairs, cols), dtype, stride=stride)
        y[count:] = float("nan")            # rows of no expert
        w = torch.randn((tokens, top_k), generator=g)
        w[place < 0] = float("nan")         # and their weights
        r = normal(g, (tokens, cols), dtype, 2.0, stride=stride) if res else None
        strides = {} if stride is None else {k: stride for k in ["y", "d"] + ["residual"] * res}
        op = H.ExpertCombine(tokens, top_k, cols, dtype, weighted=weighted, residual=res, strides=strides)
        params = [y, place.cuda()] + [w.cuda()] * weighted + [r] * res
        wd = torch.where(place >= 0, R.f64(w), 0.0) if weighted else (place >= 0).double()
        terms = rows_at(y, place) * wd[:, :, None]
        want = terms.sum(1)
        # top_k fused multiply-adds and the residual's addition, each within
        # half a unit of at most the sum of magnitudes
        mag = terms.abs().sum(1)
        if res:
            want, mag = want + R.f64(r), mag + R.f64(r).abs()
        R.close(op(*params), want, mag * (top_k + 1) * 2.0 ** -24 * 1.01, T[dtype])


@pytest.mark.parametrize("tokens, top_k, experts, cols", LAYOUTS)
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
def test_combine_grad(dtype, tokens, top_k, experts, cols):
    for i, (shard, stride) in enumerate([(False, None), (True, cols + 5), (True, cols + 8)]):
        say("combine_grad", dtype, tokens, top_k, experts, cols, shard, stride)
        g = gen(tokens + cols + 10 * i)
        _, place, order, _ = chosen(g, tokens, top_k, experts, shard)
        pairs, count = tokens * top_k, int((order >= 0).sum())
        y, dd = normal(g, (pairs, cols), dtype, stride=stride), normal(g, (tokens, cols), dtype, 0.3, stride=stride)
        y[count:] = float("nan")
        w = torch.randn((tokens, top_k), generator=g)
        w[place < 0] = float("nan")
        strides = {} if stride is None else {"dd": stride, "y": stride, "dy": stride}
        op = H.ExpertCombineGrad(tokens, top_k, cols, dtype, strides=strides)
        out = [b.empty("cuda") for b in op.results]
        out[0].fill_(7.0)
        dy, dw = op(dd, y, place.cuda(), w.cuda(), out=out)
        order = order[:count].long()
        want = R.f64(w).reshape(-1)[order][:, None] * R.f64(dd)[order // top_k]
        R.close(dy[:count], want, want.abs() * 2.0 ** -24, T[dtype])
        assert (dy[count:] == 7.0).all(), "rows of no expert changed"
        terms = rows_at(y, place) * R.f64(dd)[:, None, :]
        # a thread's chain of cols / (8 T) vectors of 8, then a wave and 4 waves
        steps = 8 * (cols // 512 + 1) + 16
        R.close(dw, terms.sum(2), steps * 2.0 ** -24 * terms.abs().sum(2), torch.float32)


def test_combine_gradients_by_differences():
    """d(sum of dd * combine) along random directions of y and weight, in f32,
    whose values are chosen so that the sums below are exact enough: the
    function is linear in each, so one difference is the derivative."""
    g = gen(5)
    tokens, top_k, experts, cols = 13, 3, 6, 40
    _, place, order, _ = chosen(g, tokens, top_k, experts, True)
    pl = place.cuda()
    y, dd = (torch.randn(s, generator=g).cuda() for s in ((tokens * top_k, cols), (tokens, cols)))
    w = torch.randn((tokens, top_k), generator=g).cuda()
    fwd = H.ExpertCombine(tokens, top_k, cols, "f32")
    op = H.ExpertCombineGrad(tokens, top_k, cols, "f32")
    out = [torch.zeros(b.dims, device="cuda") for b in op.results]
    dy, dw = op(dd, y, pl, w, out=out)
    value = lambda y, w: (R.f64(fwd(y, pl, w)) * R.f64(dd)).sum()  # noqa: E731
    vy, vw = torch.randn(y.shape, generator=g).cuda(), torch.randn(w.shape, generator=g).cuda()
    # each value is off by at most (top_k + 2) 2^-24 of its terms' magnitudes
    mag = float((rows_at(y.abs() + vy.abs(), place) * (R.f64(w).abs() + R.f64(vw).abs())[:, :, None]).sum(1).mul(R.f64(dd).abs()).sum())
    tol = 4 * (top_k + 4) * 2.0 ** -24 * mag
    assert abs(float(value(y + vy, w) - value(y, w)) - float((R.f64(dy) * R.f64(vy)).sum())) <= tol
    assert abs(float(value(y, w + vw) - value(y, w)) - float((R.f64(dw) * R.f64(vw)).sum())) <= tol
    # dispatch and combine without weights are each other's transpose
    x = torch.randn((tokens, cols), generator=g).cuda()
    z = H.ExpertDispatch(tokens, top_k, cols, "f32")(x, pl, out=torch.zeros_like(y))
    back = H.ExpertCombine(tokens, top_k, cols, "f32", weighted=False)(y, pl)
    n = int((order >= 0).sum())
    assert abs(float((R.f64(z)[:n] * R.f64(y)[:n]).sum() - (R.f64(x) * R.f64(back)).sum())) <= tol


def test_places_out_of_range_are_no_rows():
    """Whatever place holds, accesses stay in the buffers: numbers that are no
    row count as -1."""
    g = gen(8)
    tokens, top_k, cols = 9, 4, 72
    place = X.sort(torch.randint(0, 5, (tokens, top_k), generator=g, dtype=torch.int32), 5)[0]
    bad = place.clone()
    for i, v in enumerate([-2 ** 31, -2, tokens * top_k, 2 ** 31 - 1]):
        bad[2 * i, i] = v
    as_none = torch.where((bad < 0) | (bad >= tokens * top_k), -1, bad)
    x, y = normal(g, (tokens, cols), "bf16"), normal(g, (tokens * top_k, cols), "bf16")
    w = torch.randn((tokens, top_k), generator=g).cuda()
    for op, params in ((H.ExpertDispatch(tokens, top_k, cols), (x,)), (H.ExpertCombine(tokens, top_k, cols), (y,)),
                       (H.ExpertCombineGrad(tokens, top_k, cols), (x, y))):
        more = () if isinstance(op, H.ExpertDispatch) else (w,)
        got = []
        for p in (bad, as_none):
            out = [torch.zeros(b.dims, dtype=T[b.dtype], device="cuda") for b in op.results]
            op(*params, p.cuda(), *more, out=out)
            got.append(out)
        for a, b in zip(*got):
            assert torch.equal(a, b)


# --------------------------------------------------------------------------
# block scales
# --------------------------------------------------------------------------
def check_quantize(x, y, scale):
    rows, cols = x.shape
    v = R.f64(x)
    want = torch.stack([v[:, c:c + 128].abs().amax(1) for c in range(0, cols, 128)]) / 448
    R.close(scale, want, 0.0, torch.float32)
    s = X.spread_rows(scale, cols)
    q, t = R.f64(y), v / torch.where(s > 0, s, 1.0)
    # the quotient's roundings before the last one: 2^-22 covers them
    bad = ~((q - t).abs() <= t.abs() * (2.0 ** -4 + 2.0 ** -22) + 2.0 ** -10)
    assert not bad.any(), (q[bad][:4], t[bad][:4])
    assert (q.abs() <= 448).all()


@pytest.mark.parametrize("rows, cols", [(1, 11264), (1, 1), (5, 127), (4, 128), (17, 129), (33, 2048), (9, 2049), (100, 1000),
                                        (4100, 1111), (2500, 16384), (16, 20), (70000, 40), (9000, 512), (3000, 300), (333, 1024)])
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
def test_quantize(dtype, rows, cols):
    for stride in (None, cols + 1, cols + 16):
        say("quantize", dtype, rows, cols, stride)
        g = gen(rows + cols)
        x = normal(g, (rows, cols), dtype, 3.0, stride=stride)
        strides = {} if stride is None else {"x": stride, "y": stride + 1, "scale": rows + 3}
        y, scale = H.BlockQuantize(rows, cols, dtype, strides=strides)(x)
        check_quantize(x, y, scale)


def test_quantize_special_blocks():
    """Zeros, a NaN, an infinity, tiny and huge values; the blocks beside them
    are as if they were not there."""
    g = gen(3)
    x = torch.randn((6, 384), generator=g)
    x[0, 128:256] = 0
    x[1, 130] = float("nan")
    x[2, 3] = float("-inf")
    x[3, :128] *= 1e37
    x[4, 256:] *= 1e-36
    x[5, 128:256] = 0
    x[5, 255] = -1e-5
    x = x.cuda()
    y, scale = H.BlockQuantize(6, 384, "f32")(x)
    v, s = R.f64(y), scale.cpu()
    assert s[1, 0] == 0 and (v[0, 128:256] == 0).all()
    assert torch.isnan(s[1, 1]) and torch.isnan(v[1, 128:256]).all()
    assert torch.isinf(s[0, 2]) and torch.isnan(v[2, 3]) and (v[2, :3] == 0).all() and (v[2, 4:128] == 0).all()
    assert v[5, 255] == -448 and (v[5, 128:255] == 0).all()
    check_quantize(x[[0, 3, 4, 5]], y[[0, 3, 4, 5]], scale[:, [0, 3, 4, 5]])
    check_quantize(x[1:3, 256:], y[1:3, 256:], scale[2:, 1:3])


def block_operands(g, m, n, k, parts=1, spread=1.0):
    """a, b, a_scale, b_scale and the values that they stand for."""
    a = torch.randn((m, k), generator=g, dtype=torch.float64) * torch.exp(spread * torch.randn((m, 1), generator=g))
    qa, sa = X.quantize(a)
    qb, sb = zip(*[X.quantize_weight(torch.randn((n, k), generator=g, dtype=torch.float64) * max(k, 1) ** -0.5)
                   for _ in range(parts)])
    av = R.f64(qa) * X.spread_rows(sa, k)
    bv = torch.cat([R.f64(q) * X.spread_weight(s, n, k) for q, s in zip(qb, sb)])
    return [qa.cuda(), torch.cat(qb).cuda(), sa.cuda(), torch.cat(sb).cuda()], av, bv


def product_error(mag, k):
    """k products in the matrix instructions' blocks of 128 (2^-17 of their
    magnitudes) and k / 128 scaled additions of four roundings: less than
    sum_error's two units a product for k > 128.  Shorter contractions go
    through f16 exactly, with one block."""
    return R.sum_error(mag, k) + 8 * 2.0 ** -24 * mag


BLOCK_SHAPES = [(1, 16, 64), (1, 4096, 512), (3, 130, 129), (8, 512, 4096), (16, 64, 512), (17, 48, 1000), (64, 300, 2048),
                (65, 64, 64), (100, 130, 200), (129, 257, 1032), (255, 513, 328), (300, 1000, 4096), (513, 768, 144),
                (1, 1, 1), (7, 5, 3), (2, 24, 16384), (1, 8500, 384), (33, 8330, 272), (2050, 2304, 640), (1024, 1024, 1040)]


@pytest.mark.parametrize("m, n, k", BLOCK_SHAPES)
def test_block_product(m, n, k):
    g = gen(m * 7 + n * 3 + k)
    ops, av, bv = block_operands(g, m, n, k)
    z, mag = av @ bv.T, av.abs() @ bv.abs().T
    for bias, act, res, save, out in [(False, None, False, False, "bf16"), (True, "gelu", True, True, "f16"),
                                      (False, "silu", True, False, "f32")]:
        plan = H.Matmul(m, n, k, "f8e4m3", scales="blocks", out_dtype=out, mode="plan").plan()
        say("blocks", m, n, k, act, out, plan)
        op = H.Matmul(m, n, k, "f8e4m3", scales="blocks", out_dtype=out, bias=bias, activation=act, residual=res, save=save)
        extra = [normal(g, (n,), out)] * bias + [normal(g, (m, n), out)] * res
        got = op(*ops, *extra)
        want, err = z, product_error(mag, k)
        if bias:
            want = want + R.f64(extra[0])
            err = err + want.abs() * 2.0 ** -24
        if save:
            R.close(got[1], want, err, T[out])
            got = got[0]
        d = R.act(act, want)[0]
        err = 1.2 * err + (R.act_error(want) if act else 0)
        if res:
            d = d + R.f64(extra[-1])
            err = err + d.abs() * 2.0 ** -24
        R.close(got, d, err, T[out])


@pytest.mark.parametrize("m, n, k", [(1, 16, 64), (5, 130, 520), (64, 704, 1024), (70, 65, 2048), (300, 257, 392), (700, 640, 1024),
                                     (2, 4000, 512), (2060, 1024, 256)])
def test_block_gated(m, n, k):
    g = gen(m + n + k)
    ops, av, bv = block_operands(g, m, n, k, parts=2)
    z, mag = av @ bv.T, av.abs() @ bv.abs().T
    err = product_error(mag, k)
    for out, save in (("bf16", True), ("f32", False)):
        say("block gated", m, n, k, out)
        got = H.GatedFeedForward(m, n, k, "f8e4m3", scales="blocks", out_dtype=out, activation="relu", save=save)(*ops)
        if save:
            R.close(got[1], z, err, T[out])
            got = got[0]
        f, u = R.act("relu", z[:, :n])[0], z[:, n:]
        R.close(got, f * u, err[:, :n] * (u.abs() + err[:, n:]) + f.abs() * err[:, n:] + (f * u).abs() * 2.0 ** -24, T[out])


def test_block_scales_far_apart():
    """Scales whose products leave f32's range where the result is in it,
    denormal and zero ones, and a row with an infinite and one with a NaN scale."""
    g = gen(21)
    for m, n, k in ((5, 48, 512), (40, 200, 640), (300, 300, 512)):
        for out in ("bf16", "f32"):
            say("far scales", m, n, k, out)
            ops, _, _ = block_operands(g, m, n, k, spread=0.0)
            a, b, sa, sb = ops
            sa, sb = sa.clone(), sb.clone()
            sa[:, 0], sa[:, 1], sa[:, 2] = 1e30, 1e-38, 0.0
            sa[1, 1] = 1e-41                     # a denormal, beside normal ones
            sa[0, 3], sa[1, 4] = float("inf"), float("nan")
            sb[:] = torch.linspace(-4, 4, sb.shape[1], device="cuda").exp()[None, :] * 1e-3
            got = H.Matmul(m, n, k, "f8e4m3", scales="blocks", out_dtype=out)(a, b, sa, sb)
            ok = [i for i in range(m) if i not in (3, 4)]
            av = R.f64(a) * X.spread_rows(sa, k).nan_to_num(0, 0, 0)
            bv = R.f64(b) * X.spread_weight(sb, n, k)
            z, mag = av @ bv.T, av.abs() @ bv.abs().T
            R.close(got[ok], z[ok], product_error(mag, k)[ok] + 2.0 ** -140, T[out])
            assert torch.isnan(got[4].float()).all() and not torch.isfinite(got[3].float()).any()
    # 1e-30 * 1e30 for a's and b's, and the other way round
    m, n, k = 130, 128, 256
    ops, _, _ = block_operands(g, m, n, k, spread=0.0)
    for x in (1e-36, 1e36):
        sa, sb = torch.full_like(ops[2], x), torch.full_like(ops[3], 1 / x)
        got = H.Matmul(m, n, k, "f8e4m3", scales="blocks")(ops[0], ops[1], sa, sb)
        one = H.Matmul(m, n, k, "f8e4m3", scales="blocks")(ops[0], ops[1], torch.ones_like(sa), torch.ones_like(sb))
        # the scales' product is 1 to two roundings of f32, the result's rounding follows
        assert torch.isfinite(got.float()).all()
        assert ((got.float() - one.float()).abs() <= one.float().abs() * 2.0 ** -7 + 1e-30).all()


def test_block_strides():
    g = gen(31)
    for m, n, k in ((6, 40, 272), (200, 140, 300)):
        ops, av, bv = block_operands(g, m, n, k)
        z, mag = av @ bv.T, av.abs() @ bv.abs().T
        wide = []
        pads = {"a": 16, "b": 48, "a_scale": 3, "b_scale": 2}
        for t, pad in zip(ops, pads.values()):
            full = torch.full((t.shape[0], t.shape[1] + pad), float("nan"), device="cuda").to(t.dtype)
            full[:, :t.shape[1]] = t
            wide.append(full[:, :t.shape[1]])
        strides = {name: t.stride(0) for name, t in zip(pads, wide)} | {"d": n + 1}
        got = H.Matmul(m, n, k, "f8e4m3", scales="blocks", strides=strides)(*wide)
        R.close(got, z, product_error(mag, k), torch.bfloat16)


# --------------------------------------------------------------------------
# the experts' products
# --------------------------------------------------------------------------
def offsets_of(counts):
    return torch.tensor([0] + list(torch.tensor(counts).cumsum(0)), dtype=torch.int32)


# rows an expert: none, one, at and past the strips' and the tiles' sizes; rows
# that are no expert's behind them
COUNTS = {
    "one each": ([1] * 5, 0),
    "decode": ([3, 0, 1, 70, 0, 0, 8, 64], 6),
    "uneven": ([0, 130, 1, 256, 0, 129, 300, 0], 40),
    "large": ([500, 0, 257, 900], 0),
    "all to one": ([0, 0, 333, 0], 3),
    "none": ([0, 0, 0], 17),
    "many": ([(i * 7) % 5 for i in range(200)], 9),
    "a token": ([1 if i in (5, 62) else 0 for i in range(64)], 0),
}


def experts_operands(g, dtype, m, n, k, experts, parts, counts):
    """Parameters, the sums z [m, parts * n] of the rows that have an expert, and
    their magnitudes."""
    offsets = offsets_of(counts)
    ends = offsets.tolist()
    if dtype == "blocks":
        ops, av, bv = block_operands(g, m, n, k, experts * parts)
    elif dtype in ("s8", "f8e4m3"):
        (a, sa), (b, sb) = eight(g, m, k, dtype), eight(g, experts * parts * n, k, dtype)
        ops, av, bv = [a, b, sa, sb], R.f64(a) * R.f64(sa)[:, None], R.f64(b) * R.f64(sb)[:, None]
    else:
        a, b = normal(g, (m, k), dtype), normal(g, (experts * parts * n, k), dtype, max(k, 1) ** -0.5)
        a[ends[-1]:] = float("nan")       # rows of no expert
        ops, av, bv = [a, b], R.f64(a), R.f64(b)
    z, mag = torch.zeros((ends[-1], parts * n), dtype=torch.float64), torch.zeros((ends[-1], parts * n), dtype=torch.float64)
    for e in range(experts):
        rows, w = slice(ends[e], ends[e + 1]), bv[e * parts * n:(e + 1) * parts * n]
        z[rows], mag[rows] = av[rows] @ w.T, av[rows].abs() @ w.abs().T
    return ops + [offsets.cuda()], z, mag


@pytest.mark.parametrize("n, k", [(48, 64), (257, 200), (640, 1032), (130, 77)])
@pytest.mark.parametrize("counts", sorted(COUNTS))
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f8e4m3", "s8", "blocks"])
def test_experts_product(dtype, counts, n, k):
    counts, behind = COUNTS[counts]
    experts, m = len(counts), sum(counts) + behind
    eight_bits, scales = dtype in ("f8e4m3", "s8", "blocks"), "blocks" if dtype == "blocks" else None
    kind = "f8e4m3" if dtype == "blocks" else dtype
    g = gen(n + k + m)
    for parts, act, out in [(1, None, "bf16"), (1, "gelu", "f32"), (2, "relu", "f16" if dtype != "bf16" else "bf16")]:
        ops, z, mag = experts_operands(g, dtype, m, n, k, experts, parts, counts)
        if not eight_bits:
            out = "f32" if out == "f32" else dtype
        make = H.Matmul if parts == 1 else H.GatedFeedForward
        op = make(m, n, k, kind, out_dtype=out, activation=act, save=True, scales=scales, experts=experts,
                  strides={"z": parts * n + 8, "d": n + (n % 2)})
        say("experts", dtype, counts if experts < 10 else experts, n, k, parts, out, op.plan()["tile_rows"])
        res = [b.empty("cuda") for b in op.results]
        for t in res:
            t.fill_(5.0)
        d, zs = op(*ops, out=res)
        live = z.shape[0]
        err = product_error(mag, k)
        R.close(zs[:live], z, err, T[out])
        if parts == 1:
            R.close(d[:live], R.act(act, z)[0], 1.2 * err + (R.act_error(z) if act == "gelu" else 0), T[out])
        else:
            f, u = R.act("relu", z[:, :n])[0], z[:, n:]
            R.close(d[:live], f * u, err[:, :n] * (u.abs() + err[:, n:]) + f.abs() * err[:, n:] + (f * u).abs() * 2.0 ** -24, T[out])
        assert (d[live:] == 5.0).all() and (zs[live:] == 5.0).all(), "rows of no expert changed"


def test_experts_product_tiles():
    """Strips and small tiles, each with more than one tile of rows and of
    columns."""
    seen = set()
    for dtype, counts, n, k in (("bf16", [20, 90, 0, 0, 0, 7], 300, 256), ("f16", [150, 0, 400, 20], 600, 328),
                                ("blocks", [33, 90, 0, 0, 0, 0, 0], 600, 520), ("s8", [700, 90, 513, 0], 600, 520)):
        for parts in (1, 2):
            g = gen(n + parts)
            ops, z, mag = experts_operands(g, dtype, sum(counts), n, k, len(counts), parts, counts)
            kind, out = ("f8e4m3" if dtype == "blocks" else dtype), ("f16" if dtype == "f16" else "bf16")
            make = H.Matmul if parts == 1 else H.GatedFeedForward
            op = make(sum(counts), n, k, kind, out_dtype=out, activation="relu", save=True, experts=len(counts),
                      scales="blocks" if dtype == "blocks" else None)
            seen.add(op.plan()["tile_rows"])
            say("experts tiles", dtype, counts, n, k, parts, op.plan())
            R.close(op(*ops)[1], z, product_error(mag, k), T[out])
    assert seen == {64, 128}


@pytest.mark.parametrize("dtype", ["bf16", "f16", "s8", "f8e4m3", "blocks"])
@pytest.mark.parametrize("counts", [[1300, 90, 513, 700],       # 208 large tiles: whole, ragged ends as halves
                                    [2600, 90, 0, 513, 700],    # 288: 256 whole ones, the last 32 cut into halves
                                    [1024, 900, 300]])          # 160 of 256 rows: whole, ragged
def test_experts_large_tiles(dtype, counts):
    k, behind = 136, 5
    for parts in (1, 2):
        n = 4096 // parts - 8
        g = gen(sum(counts) + parts)
        m = sum(counts) + behind
        ops, z, mag = experts_operands(g, dtype, m, n, k, len(counts), parts, counts)
        make = H.Matmul if parts == 1 else H.GatedFeedForward
        half = "f16" if dtype == "f16" else "bf16"
        op = make(m, n, k, "f8e4m3" if dtype == "blocks" else dtype, out_dtype=half, activation="relu", save=True,
                  experts=len(counts), scales="blocks" if dtype == "blocks" else None)
        assert op.plan()["tile_rows"] == 256
        say("experts large", dtype, counts, n, k, parts, op.plan())
        out = [b.empty("cuda") for b in op.results]
        for t in out:
            t.fill_(5.0)
        d, zs = op(*ops, out=out)
        err = product_error(mag, k)
        R.close(zs[:z.shape[0]], z, err, T[half])
        assert (d[z.shape[0]:] == 5.0).all() and (zs[z.shape[0]:] == 5.0).all()


@pytest.mark.parametrize("dtype, out", [("bf16", "bf16"), ("f16", "f32"), ("blocks", "bf16"), ("blocks", "f32")])
@pytest.mark.parametrize("counts, n, k", [([1, 0, 1, 0], 200, 4096), ([150, 0, 40, 10], 130, 4100), ([300, 0, 1, 129], 264, 2056),
                                          ([0, 0, 3], 64, 8192)])
def test_experts_shared_contraction(dtype, out, counts, n, k):
    """Strips and small tiles whose contraction several workgroups share; the
    fold leaves rows that are no expert's as they were."""
    m, behind = sum(counts) + 4, 4
    for parts in (1, 2):
        g = gen(m + n + parts)
        ops, z, mag = experts_operands(g, dtype, m, n, k, len(counts), parts, counts)
        make = H.Matmul if parts == 1 else H.GatedFeedForward
        op = make(m, n, k, "f8e4m3" if dtype == "blocks" else dtype, out_dtype=out, activation="relu", save=True,
                  experts=len(counts), scales="blocks" if dtype == "blocks" else None)
        assert op.plan()["splits"] > 1
        say("experts shared", dtype, out, counts, n, k, parts, op.plan())
        res = [b.empty("cuda") for b in op.results]
        for t in res:
            t.fill_(5.0)
        d, zs = op(*ops, out=res)
        live = m - behind
        err = product_error(mag, k)
        R.close(zs[:live], z, err, T[out])
        want, off = R.act("relu", z[:, :n])[0], err[:, :n]
        if parts == 2:
            u = z[:, n:]
            want, off = want * u, err[:, :n] * (u.abs() + err[:, n:]) + want.abs() * err[:, n:] + (want * u).abs() * 2.0 ** -24
        R.close(d[:live], want, off, T[out])
        assert (d[live:] == 5.0).all() and (zs[live:] == 5.0).all()
        # offsets that begin past 0: rows before them too
        if dtype == "bf16":
            shifted = ops[-1] + 2
            for t in res:
                t.fill_(5.0)
            op(*ops[:-1], shifted, out=res)
            assert (res[0][:2] == 5.0).all() and (res[0][live + 2:] == 5.0).all() and not (res[0][2:live + 2] == 5.0).all()


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("counts, n, k", [([1500], 128, 200), ([900, 0, 700], 96, 328), ([5, 0, 3], 2048, 136), ([0, 0], 64, 2000),
                                          ([2000, 1], 130, 77)])
def test_experts_gradient_shared_contraction(dtype, counts, n, k):
    """da's contraction over many columns, db's over many rows, shared."""
    experts, m, live = len(counts), sum(counts) + 3, sum(counts)
    offsets = offsets_of(counts)
    g = gen(m + n)
    dd, a = normal(g, (m, n), dtype, 0.1), normal(g, (m, k), dtype)
    b = normal(g, (experts * n, k), dtype, k ** -0.5)
    for t in (dd, a):
        t[live:] = float("nan")
    op = H.MatmulGrad(m, n, k, dtype, experts=experts)
    assert op.workspace_bytes > 0 or live == 0
    say("experts gradient shared", dtype, counts, n, k, op.plan())
    out = [x.empty("cuda") for x in op.results]
    for t in out:
        t.fill_(5.0)
    da, db = op(dd, a, b, offsets.cuda(), out=out)
    want = grads_want(R.f64(dd)[:live], R.f64(a)[:live], R.f64(b), offsets.tolist(), experts)
    R.close(da[:live], want[0], R.sum_error(want[2], n), T[dtype])
    R.close(db, want[1], R.sum_error(want[3], max(counts)), T[dtype])
    assert (da[live:] == 5.0).all()


def test_experts_large_tiles_all_cut():
    """128 large tiles, every one cut into two halves."""
    counts, n, k = [1024, 768, 256], 4096, 72
    g = gen(128)
    ops, z, mag = experts_operands(g, "f16", sum(counts), n, k, 3, 1, counts)
    op = H.Matmul(sum(counts), n, k, "f16", experts=3)
    assert op.plan()["tile_rows"] == 256
    R.close(op(*ops), z, product_error(mag, k), torch.float16)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("counts", [[500, 0, 257, 130], [1, 700, 64, 0, 128]])
def test_experts_gradient_large_tiles(dtype, counts):
    experts, m, n, k = len(counts), sum(counts) + 3, 2048, 1032
    offsets, live = offsets_of(counts), sum(counts)
    for parts in (1, 2):
        cols = n // parts
        g = gen(m + parts)
        dd, a = normal(g, (m, cols), dtype, 0.1), normal(g, (m, k), dtype)
        b = normal(g, (experts * n, k), dtype, k ** -0.5)
        z = normal(g, (m, n), dtype)
        make = H.MatmulGrad if parts == 1 else H.GatedFeedForwardGrad
        op = make(m, cols, k, dtype, experts=experts, **({} if parts == 1 else dict(activation="relu")))
        assert op.plan()["tile_rows"] == 256
        say("experts gradient large", dtype, counts, parts, op.plan())
        out = [x.empty("cuda") for x in op.results]
        for t in out:
            t.fill_(5.0)
        da, db = op(*([dd, a, b] + [z] * (parts - 1) + [offsets.cuda()]), out=out)
        dz, rounded = R.f64(dd)[:live], 0.0
        if parts == 2:
            gate, u = R.f64(z)[:live, :cols], R.f64(z)[:live, cols:]
            f, df = R.act("relu", gate)
            dz = torch.cat([dz * u * df, dz * f], 1)
            rounded = dz.abs() * (R.HALF[T[dtype]] * (1 + 2.0 ** -7) + 4 * 2.0 ** -24) + R.TINY[T[dtype]]
        want = grads_want(dz, R.f64(a)[:live], R.f64(b), offsets.tolist(), experts)
        off = grads_want(dz * 0 + rounded, R.f64(a)[:live].abs(), R.f64(b).abs(), offsets.tolist(), experts)
        R.close(da[:live], want[0], R.sum_error(want[2], n) + 1.1 * off[0], T[dtype])
        R.close(db, want[1], R.sum_error(want[3], max(counts)) + 1.1 * off[1], T[dtype])
        assert (da[live:] == 5.0).all()


def grads_want(dz, a, b, ends, experts):
    """(da, db) and the magnitudes of their sums, in 64 bits."""
    wide, k = dz.shape[1], a.shape[1]
    da, db = torch.zeros((ends[-1], k), dtype=torch.float64), torch.zeros((experts * wide, k), dtype=torch.float64)
    ma, mb = torch.zeros_like(da), torch.zeros_like(db)
    for e in range(experts):
        r, w = slice(ends[e], ends[e + 1]), slice(e * wide, (e + 1) * wide)
        da[r], ma[r] = dz[r] @ b[w], dz[r].abs() @ b[w].abs()
        db[w], mb[w] = dz[r].T @ a[r], dz[r].abs().T @ a[r].abs()
    return da, db, ma, mb


@pytest.mark.parametrize("n, k", [(48, 64), (257, 200), (640, 328), (33, 77)])
@pytest.mark.parametrize("counts", sorted(COUNTS))
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_experts_gradient(dtype, counts, n, k):
    counts, behind = COUNTS[counts]
    experts, m, live = len(counts), sum(counts) + behind, sum(counts)
    offsets = offsets_of(counts)
    ends = offsets.tolist()
    half = R.HALF[T[dtype]]
    for parts, act in ((1, None), (1, "gelu"), (2, "silu")):
        g = gen(n + k + m + parts)
        dd, a = normal(g, (m, n), dtype, 0.1), normal(g, (m, k), dtype)
        b = normal(g, (experts * parts * n, k), dtype, max(k, 1) ** -0.5)
        z = normal(g, (m, parts * n), dtype)
        for t in (dd, a, z):
            t[live:] = float("nan")
        make = H.MatmulGrad if parts == 1 else H.GatedFeedForwardGrad
        op = make(m, n, k, dtype, activation=act, experts=experts)
        say("experts gradient", dtype, counts if experts < 10 else experts, n, k, parts, act, op.plan()["tile_rows"])
        out = [x.empty("cuda") for x in op.results]
        for t in out:
            t.fill_(5.0)
        da, db = op(*([dd, a, b] + [z] * (act is not None) + [offsets.cuda()]), out=out)
        v = R.f64(dd)[:live]
        rounded = 0.0
        if act is not None:
            zz = R.f64(z)[:live]
            if parts == 1:
                dz, slope = v * R.act(act, zz)[1], v.abs() * R.act_error(zz)
            else:
                gate, u = zz[:, :n], zz[:, n:]
                f, df = R.act(act, gate)
                dz = torch.cat([v * u * df, v * f], 1)
                slope = torch.cat([(v * u).abs(), v.abs()], 1) * R.act_error(gate).repeat(1, 2)
            # dz on its way into the products: one rounding of its type, the
            # activation's error and three roundings in 32 bits
            rounded = dz.abs() * (half * (1 + 2.0 ** -7) + 4 * 2.0 ** -24) + R.TINY[T[dtype]] + slope
        else:
            dz = v
        want = grads_want(dz, R.f64(a)[:live], R.f64(b), ends, experts)
        off = grads_want(dz * 0 + rounded, R.f64(a)[:live].abs(), R.f64(b).abs(), ends, experts)
        R.close(da[:live], want[0], R.sum_error(want[2], parts * n) + 1.1 * off[0], T[dtype])
        R.close(db, want[1], R.sum_error(want[3], max(counts)) + 1.1 * off[1], T[dtype])
        assert (da[live:] == 5.0).all(), "rows of no expert changed"
        for e in range(experts):
            if counts[e] == 0:
                assert (db[e * parts * n:(e + 1) * parts * n] == 0).all()


def test_experts_gradient_by_differences():
    """The gated product's gradient along random directions of a and b against
    central differences of its definition in 64 bits."""
    counts, n, k, experts = [9, 0, 20, 3], 24, 40, 4
    m = sum(counts)
    offsets = offsets_of(counts)
    ends = offsets.tolist()
    g = gen(77)
    a, b = normal(g, (m, k), "f16"), normal(g, (experts * 2 * n, k), "f16", 0.2)
    dd = normal(g, (m, n), "f16")

    def value(a, b):
        total = 0.0
        for e in range(experts):
            r = slice(ends[e], ends[e + 1])
            z = a[r] @ b[e * 2 * n:(e + 1) * 2 * n].T
            total += (R.act("silu", z[:, :n])[0] * z[:, n:] * R.f64(dd)[r]).sum()
        return float(total)

    # z in f16: its rounding moves the slopes by 2^-11 of them
    _, z = H.GatedFeedForward(m, n, k, "f16", save=True, experts=experts)(a, b, offsets.cuda())
    da, db = H.GatedFeedForwardGrad(m, n, k, "f16", experts=experts)(dd, a, b, z, offsets.cuda())
    x, w = R.f64(a), R.f64(b)
    va, vb = torch.randn(x.shape, generator=g).double(), torch.randn(w.shape, generator=g).double()
    for grad, at in ((da, lambda h: value(x + h * va, w)), (db, lambda h: value(x, w + h * vb))):
        v = va if grad is da else vb
        got, want = float((R.f64(grad) * v).sum()), (at(1e-4) - at(-1e-4)) / 2e-4
        # every term may be off by the roundings of z, dz and the gradient: 4 of
        # 2^-11, of the terms' magnitudes
        assert abs(got - want) <= 4 * 2.0 ** -11 * float((R.f64(grad).abs() * v.abs()).sum()) * 2, (got, want)


def test_offsets_that_skip_rows():
    """Rows before the first expert's and between none: offsets that begin past
    0 name the rows of a shard."""
    g = gen(91)
    n, k, experts = 96, 128, 3
    a, b = normal(g, (60, k), "bf16"), normal(g, (experts * n, k), "bf16", 0.1)
    offsets = torch.tensor([7, 20, 20, 41], dtype=torch.int32)
    op = H.Matmul(60, n, k, "bf16", out_dtype="f32", experts=experts)
    d = op(a, b, offsets.cuda(), out=torch.full((60, n), 3.0, device="cuda"))
    assert (d[:7] == 3.0).all() and (d[41:] == 3.0).all()
    for e, (lo, hi) in enumerate([(7, 20), (20, 20), (20, 41)]):
        w = R.f64(b)[e * n:(e + 1) * n]
        x = R.f64(a)[lo:hi]
        R.close(d[lo:hi], x @ w.T, R.sum_error(x.abs() @ w.abs().T, k), torch.float32)


def test_offsets_out_of_range_stay_in_the_buffers():
    """Offsets that decrease or leave 0 .. m: rows are held to the buffer.  Which
    results they give is not defined; memory around the results is unchanged."""
    g = gen(92)
    m, n, k, experts = 70, 64, 64, 4
    a, b = normal(g, (m, k), "bf16"), normal(g, (experts * n, k), "bf16", 0.1)
    around = torch.full((m + 200, n), 3.0, device="cuda", dtype=torch.bfloat16)
    op = H.Matmul(m, n, k, "bf16", experts=experts)
    for bad in ([-5, 10, 2 ** 31 - 1, 3, 70], [60, 20, 0, -1, 1000], [71, 72, 73, 74, 75], [-2 ** 31] * 5):
        op(a, b, torch.tensor(bad, dtype=torch.int32).cuda(), out=around[100:100 + m])
        torch.cuda.synchronize()
        assert (around[:100] == 3.0).all() and (around[100 + m:] == 3.0).all()


def test_no_rows_and_no_columns():
    z = lambda *s: torch.zeros(s, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    off = torch.zeros(4, dtype=torch.int32, device="cuda")
    assert H.Matmul(0, 8, 16, experts=3)(z(0, 16), z(24, 16), off).shape == (0, 8)
    assert H.Matmul(5, 0, 16, experts=3)(z(5, 16), z(0, 16), off).shape == (5, 0)
    d = H.Matmul(2, 8, 0, experts=3)(z(2, 0), z(24, 0), torch.tensor([0, 1, 2, 2], dtype=torch.int32, device="cuda"))
    assert (d == 0).all()
    da, db = H.MatmulGrad(0, 8, 16, experts=3)(z(0, 8), z(0, 16), z(24, 16), off)
    assert da.shape == (0, 16) and (db == 0).all()
    da, db = H.MatmulGrad(4, 0, 16, experts=3)(z(4, 0), z(4, 16), z(0, 16),
                                               torch.tensor([0, 4, 4, 4], dtype=torch.int32, device="cuda"))
    assert (da == 0).all() and db.shape == (0, 16)
    da, db = H.MatmulGrad(4, 8, 0, experts=3)(z(4, 8), z(4, 0), z(24, 0), off)
    assert da.shape == (4, 0) and db.shape == (24, 0)
    place = torch.zeros((0, 2), dtype=torch.int32, device="cuda")
    assert H.ExpertDispatch(0, 2, 8)(z(0, 8), place).shape == (0, 8)
    assert H.ExpertCombine(0, 2, 8)(z(0, 8), place, torch.zeros((0, 2), device="cuda")).shape == (0, 8)
    place = torch.tensor([[0, 1], [-1, 2]], dtype=torch.int32, device="cuda")
    dy, dw = H.ExpertCombineGrad(2, 2, 0)(z(2, 0), z(4, 0), place, torch.ones((2, 2), device="cuda"))
    assert dy.shape == (4, 0) and (dw == 0).all()
    y, scale = H.BlockQuantize(0, 8)(z(0, 8))
    assert y.shape == (0, 8) and scale.shape == (1, 0)
    y, scale = H.BlockQuantize(3, 0)(z(3, 0))
    assert y.shape == (3, 0) and scale.shape == (0, 3)


# --------------------------------------------------------------------------
# together, as they are used
# --------------------------------------------------------------------------
class Layer:
    """A layer of experts, forward and backward, on fixed buffers."""

    def __init__(self, tokens, top_k, experts, hidden, inner, g, stream=None):
        self.x = normal(g, (tokens, hidden), "bf16")
        self.res = normal(g, (tokens, hidden), "bf16")
        self.w_up = normal(g, (experts * 2 * inner, hidden), "bf16", hidden ** -0.5)
        self.w_down = normal(g, (experts * hidden, inner), "bf16", inner ** -0.5)
        self.ids = torch.randint(0, experts, (tokens, top_k), generator=g, dtype=torch.int32).cuda()
        self.weight = torch.rand((tokens, top_k), generator=g).cuda()
        self.dd = normal(g, (tokens, hidden), "bf16", 0.1)
        pairs = tokens * top_k
        bind = lambda op, *p: op.bind(*p, stream=stream)  # noqa: E731
        self.sort = bind(H.ExpertSort(tokens, top_k, experts), self.ids)
        place, order, offsets = self.sort.results
        self.send = bind(H.ExpertDispatch(tokens, top_k, hidden), self.x, place)
        self.up = bind(H.GatedFeedForward(pairs, inner, hidden, save=True, experts=experts), self.send.results, self.w_up, offsets)
        h, z = self.up.results
        self.down = bind(H.Matmul(pairs, hidden, inner, experts=experts), h, self.w_down, offsets)
        self.back = bind(H.ExpertCombine(tokens, top_k, hidden, residual=True), self.down.results, place, self.weight, self.res)
        self.dback = bind(H.ExpertCombineGrad(tokens, top_k, hidden), self.dd, self.down.results, place, self.weight)
        dy, self.dweight = self.dback.results
        self.ddown = bind(H.MatmulGrad(pairs, hidden, inner, experts=experts), dy, h, self.w_down, offsets)
        dh, self.dw_down = self.ddown.results
        self.dup = bind(H.GatedFeedForwardGrad(pairs, inner, hidden, experts=experts), dh, self.send.results, self.w_up, z, offsets)
        drows, self.dw_up = self.dup.results
        self.dsend = bind(H.ExpertCombine(tokens, top_k, hidden, weighted=False), drows, place)
        self.launches = [self.sort, self.send, self.up, self.down, self.back, self.dback, self.ddown, self.dup, self.dsend]
        self.results = [self.back.results, self.dweight, self.dw_down, self.dw_up, self.dsend.results]

    def run(self, stream=None):
        for launch in self.launches:
            launch(stream)


def layer_want(l, experts, inner):
    """The same by torch's autograd in 64 bits on the CPU, token by token."""
    x, up, down, w = (R.f64(t).requires_grad_() for t in (l.x, l.w_up, l.w_down, l.weight))
    hidden = x.shape[1]
    rows = []
    for t in range(x.shape[0]):
        y = R.f64(l.res)[t]
        for j in range(w.shape[1]):
            e = int(l.ids[t, j])
            z = up[e * 2 * inner:(e + 1) * 2 * inner] @ x[t]
            y = y + w[t, j] * (down[e * hidden:(e + 1) * hidden] @ (torch.nn.functional.silu(z[:inner]) * z[inner:]))
        rows.append(y)
    y = torch.stack(rows)
    (y * R.f64(l.dd)).sum().backward()
    return [y.detach(), w.grad, down.grad, up.grad, x.grad]


def test_a_layer_of_experts():
    """Sort, dispatch, both products, combine and all their gradients in a row.
    Each of the intermediate arrays is rounded to bf16 (8 of them follow one
    another on the longest way), so relative to the norm of the result the
    errors stay below 8 * 2^-8."""
    tokens, top_k, experts, hidden, inner = 40, 2, 5, 64, 48
    l = Layer(tokens, top_k, experts, hidden, inner, gen(13))
    l.run()
    for k, (got, want) in enumerate(zip(l.results, layer_want(l, experts, inner))):
        off = float((R.f64(got) - want).norm() / want.norm())
        assert off < 8 * 2.0 ** -8, (k, off)


def test_a_layer_in_a_graph_and_on_two_streams():
    """Replays read new choices and inputs; two layers run on two streams at
    once, each with its own buffers and workspaces."""
    size = (700, 4, 12, 256, 200)
    streams = [torch.cuda.Stream() for _ in range(2)]
    layers = [Layer(*size, gen(i)) for i in range(2)]
    layers[0].run(), layers[1].run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        layers[0].run()
    g = gen(50)
    for turn in range(4):
        layers[0].x.copy_(torch.randn(layers[0].x.shape, generator=g).to(torch.bfloat16))
        # in the last turn one expert gets everything
        ids = torch.randint(0, 12, layers[0].ids.shape, generator=g, dtype=torch.int32)
        layers[0].ids.copy_(ids * 0 + 5 if turn == 3 else ids)
        layers[0].run()
        want = [t.clone() for t in layers[0].results]
        for t in layers[0].results:
            t.zero_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for k, (t, v) in enumerate(zip(layers[0].results, want)):
            assert torch.equal(t, v), (turn, k)
    wants = []
    for l in layers:
        l.run()
        torch.cuda.synchronize()
        wants.append([t.clone() for t in l.results])
    for _ in range(5):
        for l, s in zip(layers, streams):
            l.run(s)
    torch.cuda.synchronize()
    for l, w in zip(layers, wants):
        for t, v in zip(l.results, w):
            assert torch.equal(t, v)


def test_a_layer_served_with_block_scales():
    """Rows quantised, sent with their scales, both products by expert in e4m3,
    against the same values in 64 bits."""
    tokens, top_k, experts, hidden, inner = 30, 3, 6, 384, 200
    g = gen(17)
    pairs = tokens * top_k
    x = normal(g, (tokens, hidden), "bf16")
    ids = torch.randint(0, experts, (tokens, top_k), generator=g, dtype=torch.int32)
    weight = torch.rand((tokens, top_k), generator=g).cuda()
    ups = [X.quantize_weight(torch.randn((inner, hidden), generator=g).double() * hidden ** -0.5) for _ in range(2 * experts)]
    downs = [X.quantize_weight(torch.randn((hidden, inner), generator=g).double() * inner ** -0.5) for _ in range(experts)]
    cat = lambda v: (torch.cat([q for q, _ in v]).cuda(), torch.cat([s for _, s in v]).cuda())  # noqa: E731
    (w_up, s_up), (w_down, s_down) = cat(ups), cat(downs)
    place, order, offsets = H.ExpertSort(tokens, top_k, experts)(ids.cuda())
    q, s = H.BlockQuantize(tokens, hidden)(x)
    rows, rows_s = H.ExpertDispatch(tokens, top_k, hidden, "f8e4m3", scales="blocks")(q, place, s)
    h = H.GatedFeedForward(pairs, inner, hidden, "f8e4m3", scales="blocks", experts=experts)(rows, w_up, rows_s, s_up, offsets)
    hq, hs = H.BlockQuantize(pairs, inner)(h)
    y = H.Matmul(pairs, hidden, inner, "f8e4m3", scales="blocks", experts=experts)(hq, w_down, hs, s_down, offsets)
    d = H.ExpertCombine(tokens, top_k, hidden)(y, place, weight)
    xv = R.f64(q) * X.spread_rows(s, hidden)
    hv = R.f64(hq) * X.spread_rows(hs, inner)
    want_h, want_d = torch.zeros((pairs, inner), dtype=torch.float64), torch.zeros((tokens, hidden), dtype=torch.float64)
    for p in range(pairs):
        t, e, r = p // top_k, int(ids[p // top_k, p % top_k]), int(place[p // top_k, p % top_k])
        gate, up = (R.f64(ups[2 * e + i][0]) * X.spread_weight(ups[2 * e + i][1], inner, hidden) @ xv[t] for i in (0, 1))
        want_h[r] = torch.nn.functional.silu(gate) * up
        want_d[t] += float(weight[t, p % top_k]) * (R.f64(downs[e][0]) * X.spread_weight(downs[e][1], hidden, inner) @ hv[r])
    # one rounding to bf16, and below 2^-9 of the norm for the rest
    assert float((R.f64(h) - want_h).norm() / want_h.norm()) < 2.0 ** -8
    # y's rounding, then d's
    assert float((R.f64(d) - want_d).norm() / want_d.norm()) < 2 * 2.0 ** -8


def test_equal_calls_give_equal_bits():
    l = Layer(300, 4, 9, 256, 136, gen(23))
    l.run()
    want = [t.clone() for t in l.results]
    for _ in range(3):
        l.run()
    for t, v in zip(l.results, want):
        assert torch.equal(t, v)


def test_launch_refusals():
    op = H.Matmul(8, 16, 32, experts=2)
    a, b = torch.zeros((8, 32), dtype=torch.bfloat16, device="cuda"), torch.zeros((32, 32), dtype=torch.bfloat16, device="cuda")
    off = torch.zeros(3, dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError, match="offsets must be a GPU tensor"):
        op(a, b, off.long())
    with pytest.raises(ValueError, match="offsets must be a GPU tensor"):
        op(a, b, off[:2])
    with pytest.raises(ValueError, match="expected 3 parameters"):
        op(a, b)
    with pytest.raises(ValueError, match="b must be a GPU tensor"):
        op(a, b[:16], off)
    sort = H.ExpertSort(4, 2, 3)
    with pytest.raises(ValueError, match="expert must be a GPU tensor"):
        sort(torch.zeros((4, 2), dtype=torch.int64, device="cuda"))
    x = torch.zeros((4, 16), dtype=torch.bfloat16, device="cuda")
    place = torch.zeros((4, 2), dtype=torch.int32, device="cuda")
    with pytest.raises(H.FusionError, match="overlaps"):
        H.ExpertCombine(4, 1, 16, weighted=False)(x, torch.zeros((4, 1), dtype=torch.int32, device="cuda"), out=x)
    big = H.ExpertSort(70000, 4, 64)
    assert big.workspace_bytes > 0
    ids = torch.zeros((70000, 4), dtype=torch.int32, device="cuda")
    outs = [r.empty("cuda") for r in big.results]
    with pytest.raises(H.FusionError, match="needs a workspace"):
        big.launch_ptrs([ids.data_ptr()], [t.data_ptr() for t in outs])
    big.launch_noalloc_ptrs([ids.data_ptr()], [t.data_ptr() for t in outs], torch.cuda.current_stream().cuda_stream)
    torch.cuda.synchronize()
    same(outs, X.sort(ids.cpu(), 64))
    assert place is not None
