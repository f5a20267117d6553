"""The operators on the GPU against plain 64-bit forms of their definitions:
types, directions, the sizes at which a kernel, a tile or a split changes, odd
lengths, row strides, empty arrays, special values, streams and graphs."""
import math

import pytest
import torch

import compiler_hlo_amd as H
import operators_reference as R

pytestmark = pytest.mark.gpu

T = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16, "s8": torch.int8,
     "f8e4m3": torch.float8_e4m3fn}


def gen(seed):
    return torch.Generator().manual_seed(seed)


def normal(g, shape, dtype, sigma=1.0, stride=None, fill=float("nan")):
    """A GPU tensor; with `stride`, a view of rows further apart, the gaps NaN
    (a kernel that reads a gap into a result shows it)."""
    v = (torch.randn(shape, generator=g) * sigma).to(T[dtype])
    if stride is None:
        return v.cuda()
    rows, cols = shape
    full = torch.full((max(1, rows) * stride,), fill).to(T[dtype]).cuda()
    view = full.as_strided((rows, cols), (stride, 1))
    view.copy_(v.cuda())
    return view


def eight(g, rows, k, dtype):
    """(values, scales): rows in 8 bits."""
    x = torch.randn((rows, k), generator=g)
    top = {"s8": 127.0, "f8e4m3": 448.0}[dtype]
    s = x.abs().amax(1).clamp(min=1e-6) / top if k else torch.ones(rows)
    q = x / s[:, None]
    q = q.round().clamp(-127, 127).to(torch.int8) if dtype == "s8" else q.clamp(-448, 448).to(T[dtype])
    return q.cuda(), s.float().cuda()


def say(*a):
    print(*a, flush=True)


# --------------------------------------------------------------------------
# norm
# --------------------------------------------------------------------------
def norm_sum_error(cols):
    """Relative error of a sum of squares: at most cols / 1024 + 64 roundings
    follow one another in a thread, its wave and the row."""
    return (cols / 1024 + 64) * 2.0 ** -24


def check_norm(x, weight, residual, out, eps, got):
    h = R.f64(x) + (R.f64(residual) if residual is not None else 0)
    cols = h.shape[1]
    rstd = (h.square().mean(1) + eps).rsqrt()
    rel = norm_sum_error(cols) / 2 + 4 * 2.0 ** -24
    h_err = h.abs() * 2.0 ** -24                      # the sum x + residual in 32 bits
    y = h * rstd[:, None] * R.f64(weight)
    y_err = y.abs() * (rel + 4 * 2.0 ** -24)
    got = list(got)
    if out in ("s8", "f8e4m3"):
        top = {"s8": 127.0, "f8e4m3": 448.0}[out]
        scale = y.abs().amax(1) / top
        R.close(got[1], scale, scale * (rel + 8 * 2.0 ** -24), torch.float32)
        gs = R.f64(got[1])[:, None]
        q, want = R.f64(got[0]), y / torch.where(gs > 0, gs, 1.0)
        half = 0.5 if out == "s8" else want.abs() * 2.0 ** -4 + 2.0 ** -10
        bad = (q - want).abs() > half + y_err / torch.where(gs > 0, gs, 1.0) + want.abs() * 2.0 ** -22
        assert not bad.any(), (q[bad][:4], want[bad][:4])
        assert (q.abs() <= top).all()
        got = got[:1] + got[2:]
    else:
        R.close(got[0], y, y_err, T[out])
    if residual is not None:
        R.close(got[1], h, h_err, x.dtype)
    R.close(got[-1], rstd, rstd * rel, torch.float32)


LENGTHS = [1, 7, 8, 64, 511, 512, 513, 1024, 1025, 2047, 2048, 4096, 4104, 8192, 16384, 16391, 32768, 40000]


@pytest.mark.parametrize("cols", LENGTHS)
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
def test_norm(dtype, cols):
    for k, (rows, out, res, wide) in enumerate([(1, dtype, False, False), (5, "f8e4m3", True, True),
                                                (6, "s8", False, False), (9, dtype, True, True)]):
        say("norm", dtype, rows, cols, out, res)
        g = gen(100 * cols + k)
        x = normal(g, (rows, cols), dtype, 1.5)
        w = normal(g, (cols,), "f32" if wide else dtype, 0.5)
        r = normal(g, (rows, cols), dtype, 2.0) if res else None
        op = H.RmsNorm(rows, cols, dtype, residual=res, out_dtype=out, weight_dtype="f32" if wide else dtype, eps=1e-5)
        check_norm(x, w, r, out, 1e-5, op(*([x, w] + ([r] if res else []))))


@pytest.mark.parametrize("cols, stride", [(512, 520), (512, 515), (333, 400), (4096, 12288), (20, 21)])
@pytest.mark.parametrize("out", ["bf16", "f8e4m3"])
def test_norm_row_strides(cols, stride, out):
    g = gen(cols + stride)
    rows = 11
    x, r = normal(g, (rows, cols), "bf16", stride=stride), normal(g, (rows, cols), "bf16", stride=stride + 8)
    w = normal(g, (cols,), "bf16")
    op = H.RmsNorm(rows, cols, "bf16", residual=True, out_dtype=out,
                   strides={"x": stride, "residual": stride + 8, "y": stride, "stream": stride})
    got = op(x, w, r)
    assert got[0].stride(0) == stride
    check_norm(x, w, r, out, 1e-5, got)


def test_norm_special_rows():
    """Rows of zeros, of tiny and huge values, with infinities and NaN; every
    other row is as if they were not there."""
    g = gen(7)
    rows, cols = 8, 1000
    x = torch.randn((rows, cols), generator=g)
    x[1] = 0.0
    x[2] = 1e-30 * torch.sign(x[2])
    x[3] *= 1e18
    x[4, 17] = float("inf")
    x[5, 3] = float("nan")
    x = x.cuda()
    w = torch.ones(cols, device="cuda")
    q, scale, rstd = H.RmsNorm(rows, cols, "f32", out_dtype="f8e4m3", eps=0.0)(x, w)
    ok = [0, 2, 3, 6, 7]
    check_norm(x[ok], w, None, "f8e4m3", 0.0, [t[ok] for t in (q, scale, rstd)])
    assert torch.isnan(scale[4]) and torch.isnan(scale[5])
    q, scale, rstd = H.RmsNorm(rows, cols, "f32", out_dtype="s8", eps=1e-5)(x, w)
    assert scale[1] == 0 and (q[1] == 0).all() and abs(float(rstd[1]) - 1e-5 ** -0.5) < 1e-4
    y, _ = H.RmsNorm(rows, cols, "f32", eps=1e-5)(x, w)
    assert (y[1] == 0).all() and torch.isnan(y[5]).all() and torch.isnan(y[4, 17]) and (y[4, 18:] == 0).all()


def norm_grad_want(dy, h, w, rstd, ds):
    dy, h, w, rstd = map(R.f64, (dy, h, w, rstd))
    xh, g = h * rstd[:, None], dy * w
    cols = h.shape[1]
    c = (g * xh).mean(1, keepdim=True) if cols else 0
    dx = (g - xh * c) * rstd[:, None]
    err = (g.abs() + xh.abs() * (g * xh).abs().mean(1, keepdim=True) * (1 + cols / 1024 + 64)) * rstd[:, None] * 8 * 2.0 ** -24
    if ds is not None:
        dx = dx + R.f64(ds)
        err = err + dx.abs() * 2.0 ** -24
    terms = dy * xh
    return dx, err, terms.sum(0), (h.shape[0] + 8) * 2.0 ** -24 * terms.abs().sum(0)


@pytest.mark.parametrize("cols", LENGTHS)
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
def test_norm_grad(dtype, cols):
    for k, (rows, ds, wide) in enumerate([(1, False, False), (37, True, True)]):
        say("norm_grad", dtype, rows, cols)
        g = gen(300 * cols + k)
        dy, h = normal(g, (rows, cols), dtype, 0.3), normal(g, (rows, cols), dtype, 2.0)
        w = normal(g, (cols,), "f32" if wide else dtype)
        rstd = (R.f64(h).square().mean(1) + 1e-5).rsqrt().float().cuda()
        s = normal(g, (rows, cols), dtype, 0.3) if ds else None
        op = H.RmsNormGrad(rows, cols, dtype, stream_grad=ds, weight_dtype="f32" if wide else dtype)
        dx, dw = op(*([dy, h, w, rstd] + ([s] if ds else [])))
        want, err, wdw, edw = norm_grad_want(dy, h, w, rstd, s)
        R.close(dx, want, err, T[dtype])
        R.close(dw, wdw, edw, torch.float32)


def test_norm_grad_many_rows_and_strides():
    """More rows than groups, so that a group takes several; strided rows."""
    for rows, cols, stride in ((9001, 96, 96), (5003, 1032, 1048), (1500, 4100, 4101)):
        say("norm_grad", rows, cols, stride)
        g = gen(rows)
        dy, h = normal(g, (rows, cols), "bf16", stride=stride), normal(g, (rows, cols), "bf16", stride=stride)
        w = normal(g, (cols,), "bf16")
        rstd = (R.f64(h).square().mean(1) + 1e-5).rsqrt().float().cuda()
        op = H.RmsNormGrad(rows, cols, "bf16", strides={"dy": stride, "h": stride, "dx": stride + 4})
        dx, dw = op(dy, h, w, rstd)
        want, err, wdw, edw = norm_grad_want(dy, h, w, rstd, None)
        R.close(dx, want, err, torch.bfloat16)
        R.close(dw, wdw, edw, torch.float32)
        assert torch.equal(dw, op(dy, h, w, rstd)[1]), "the weight's gradient changes from run to run"


def test_norm_no_rows():
    x, w = torch.empty((0, 64), dtype=torch.bfloat16, device="cuda"), torch.ones(64, dtype=torch.bfloat16, device="cuda")
    y, rstd = H.RmsNorm(0, 64, "bf16")(x, w)
    assert y.shape == (0, 64) and rstd.shape == (0,)
    _, dw = H.RmsNormGrad(0, 64, "bf16")(x, x, w, rstd)
    assert (dw == 0).all()


# --------------------------------------------------------------------------
# products
# --------------------------------------------------------------------------
def operands(g, m, n, k, dtype, strides=None):
    strides = strides or {}
    if dtype in ("s8", "f8e4m3"):
        (a, sa), (b, sb) = eight(g, m, k, dtype), eight(g, n, k, dtype)
        return [a, b, sa, sb]
    return [normal(g, (m, k), dtype, 1.0, strides.get("a")), normal(g, (n, k), dtype, max(k, 1) ** -0.5, strides.get("b"))]


def sums(ops):
    """The 64-bit product and the sum of magnitudes of its terms."""
    a, b = R.f64(ops[0]), R.f64(ops[1])
    z, mag = a @ b.T, a.abs() @ b.abs().T
    if len(ops) > 2:
        s = R.f64(ops[2])[:, None] * R.f64(ops[3])
        z, mag = z * s, mag * s
    return z, mag


def check_matmul(ops, extra, got, out, activation, save):
    z, mag = sums(ops)
    k = ops[0].shape[1]
    err = R.sum_error(mag, k) + 4 * 2.0 ** -24 * mag
    i = 0
    if extra.get("bias") is not None:
        z = z + R.f64(extra["bias"])
        err = err + z.abs() * 2.0 ** -24
    if save:
        R.close(got[1], z, err, T[out])
        got = got[0]
    d = R.act(activation, z)[0]
    err = 1.2 * err + (R.act_error(z) if activation in ("silu", "gelu") else 0)
    if extra.get("residual") is not None:
        d = d + R.f64(extra["residual"])
        err = err + d.abs() * 2.0 ** -24
    R.close(got, d, err, T[out])


# rows at which the kernel changes (16, 32, 64 | tiles), columns inside and
# past a tile, contractions of whole and ragged steps
SHAPES = [(1, 16, 64), (1, 4096, 512), (3, 33, 96), (16, 64, 512), (17, 48, 1000), (32, 528, 2048), (33, 40, 640),
          (64, 256, 4096), (65, 64, 64), (100, 130, 200), (128, 128, 128), (129, 257, 1032), (255, 513, 328),
          (300, 1000, 4096), (513, 768, 72), (1, 1, 1), (7, 5, 3), (70, 70, 70), (2, 24, 16384), (130, 128, 8192)]


@pytest.mark.parametrize("m, n, k", SHAPES)
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f8e4m3", "s8"])
def test_matmul(dtype, m, n, k):
    for i, (bias, act, res, save, out) in enumerate([(False, None, False, False, "f32"),
                                                     (True, "gelu", True, True, "bf16"),
                                                     (False, "silu", True, False, "f16"),
                                                     (True, "relu", False, True, "f32")]):
        say("matmul", dtype, m, n, k, bias, act, res, save, out)
        g = gen(m * 7 + n * 3 + k + i)
        ops = operands(g, m, n, k, dtype)
        extra = {}
        if bias:
            extra["bias"] = normal(g, (n,), out)
        if res:
            extra["residual"] = normal(g, (m, n), out)
        op = H.Matmul(m, n, k, dtype, out_dtype=out, bias=bias, activation=act, residual=res, save=save)
        check_matmul(ops, extra, op(*ops, *extra.values()), out, act, save)


@pytest.mark.parametrize("m, n, k", [(5, 3000, 512), (2100, 2304, 256), (3000, 4352, 72)])
def test_matmul_large_tiles(m, n, k):
    """Enough tiles for the larger tile (and, for 5 rows, for 8 waves)."""
    for dtype in ("bf16", "f8e4m3"):
        say("matmul", dtype, m, n, k, H.Matmul(m, n, k, dtype, mode="plan").plan())
        ops = operands(gen(m + n), m, n, k, dtype)
        check_matmul(ops, {}, H.Matmul(m, n, k, dtype, out_dtype="f32")(*ops), "f32", None, False)


@pytest.mark.parametrize("strides", [{"a": 264, "b": 272, "d": 104, "residual": 112},
                                     {"a": 261, "b": 300, "d": 101, "residual": 103},
                                     {"a": 264, "d": 101}, {"b": 1024, "residual": 200}])
@pytest.mark.parametrize("m", [4, 70, 200])
@pytest.mark.parametrize("k", [256, 200, 251])
def test_matmul_row_strides(m, k, strides):
    n = 96
    g = gen(m + k)
    a, b = normal(g, (m, k), "bf16", stride=strides.get("a")), normal(g, (n, k), "bf16", 0.1, strides.get("b"))
    r = normal(g, (m, n), "bf16", stride=strides.get("residual"))
    op = H.Matmul(m, n, k, "bf16", residual=True, strides=strides)
    got = op(a, b, r)
    assert got.stride(0) == strides.get("d", n)
    check_matmul([a, b], {"residual": r}, got, "bf16", None, False)


def test_matmul_writes_only_its_window():
    """The gaps of a strided result keep what they held."""
    for m in (5, 90):
        base = torch.full((m, 160), 7.0, dtype=torch.bfloat16, device="cuda")
        g = gen(m)
        a, b = normal(g, (m, 128), "bf16"), normal(g, (70, 128), "bf16")
        H.Matmul(m, 70, 128, "bf16", strides={"d": 160})(a, b, out=base[:, 32:102])
        assert (base[:, :32] == 7).all() and (base[:, 102:] == 7).all()
        check_matmul([a, b], {}, base[:, 32:102], "bf16", None, False)


def test_matmul_empty():
    half = dict(dtype=torch.bfloat16, device="cuda")
    assert H.Matmul(0, 8, 16)(torch.empty((0, 16), **half), torch.ones((8, 16), **half)).shape == (0, 8)
    assert H.Matmul(3, 0, 16)(torch.ones((3, 16), **half), torch.empty((0, 16), **half)).shape == (3, 0)
    for m in (3, 80):
        bias = torch.arange(8, **half)
        d = H.Matmul(m, 8, 0, bias=True)(torch.empty((m, 0), **half), torch.empty((8, 0), **half), bias)
        assert torch.equal(d, bias.expand(m, 8))
    da, db = H.MatmulGrad(0, 8, 16)(torch.empty((0, 8), **half), torch.empty((0, 16), **half), torch.ones((8, 16), **half))
    assert da.shape == (0, 16) and (db == 0).all()
    da, db, dbias = H.MatmulGrad(3, 0, 16, bias=True)(torch.empty((3, 0), **half), torch.ones((3, 16), **half),
                                                      torch.empty((0, 16), **half))
    assert (da == 0).all() and db.shape == (0, 16) and dbias.shape == (0,)
    da, db = H.MatmulGrad(3, 8, 0)(torch.ones((3, 8), **half), torch.empty((3, 0), **half), torch.empty((8, 0), **half))
    assert da.shape == (3, 0) and db.shape == (8, 0)
    x = torch.empty((0, 16), **half)
    da, db = H.GatedFeedForwardGrad(0, 8, 16)(torch.empty((0, 8), **half), x, torch.ones((16, 16), **half),
                                              torch.empty((0, 16), **half))
    assert da.shape == (0, 16) and (db == 0).all()


def test_matmul_infinities_and_nan_stay_in_their_rows():
    for m in (40, 200):
        g = gen(m)
        a, b = normal(g, (m, 192), "bf16"), normal(g, (96, 192), "bf16")
        a[3, 5], a[9, 0], b[11, 7] = float("inf"), float("nan"), float("-inf")
        d = H.Matmul(m, 96, 192, "bf16", out_dtype="f32")(a, b)
        rows = torch.ones(m, dtype=torch.bool)
        rows[[3, 9]] = False
        cols = torch.ones(96, dtype=torch.bool)
        cols[11] = False
        assert torch.isnan(d[9]).all() and not torch.isfinite(d[3]).any() and not torch.isfinite(d[:, 11]).any()
        assert torch.isfinite(d[rows.cuda()][:, cols.cuda()]).all()


@pytest.mark.parametrize("act", ["relu", "gelu", "silu"])
def test_activation_limits(act):
    """act and act' at 0, +-inf, NaN and far values, through a product with
    one: a 1 x 1 contraction whose sum is the value itself."""
    v = torch.tensor([0.0, -0.0, 1e-3, -1e-3, 5.0, -5.0, 40.0, -40.0, 1e30, -1e30, float("inf"), float("-inf"),
                      float("nan")], dtype=torch.bfloat16, device="cuda")
    n = v.numel()
    one = torch.ones((n, 1), dtype=torch.bfloat16, device="cuda")
    d, z = H.Matmul(1, n, 1, "bf16", bias=True, activation=act, save=True, out_dtype="bf16")(
        torch.zeros((1, 1), dtype=torch.bfloat16, device="cuda"), one, v)
    assert torch.equal(torch.nan_to_num(z[0], nan=-77.0), torch.nan_to_num(v, nan=-77.0))
    x = R.f64(v)
    want, slope = R.act(act, x)
    want[10], want[11], slope[8], slope[9], slope[10], slope[11] = math.inf, 0.0, 1.0, 0.0, 1.0, 0.0
    if act != "relu":
        want[9] = 0.0
    fine = torch.isfinite(want)
    R.close(d[0][fine.cuda()], want[fine], R.act_error(x[fine].clamp(-100, 100)), torch.bfloat16)
    assert d[0, 10] == math.inf and torch.isnan(d[0, 12])
    dd = torch.ones((1, n), dtype=torch.bfloat16, device="cuda")
    dbias = H.MatmulGrad(1, n, 1, "bf16", bias=True, activation=act)(dd, one[:1], one, v[None])[2]
    R.close(dbias[:12], slope[:12], R.act_error(x[:12].clamp(-100, 100)), torch.float32)


def grad_want(dd, z, act, gated):
    dd = R.f64(dd)
    if gated:
        n = dd.shape[1]
        gate, up = R.f64(z)[:, :n], R.f64(z)[:, n:]
        f, df = R.act(act, gate)
        e = R.act_error(gate)
        return torch.cat([dd * up * df, dd * f], 1), torch.cat([(dd * up).abs() * e, dd.abs() * e], 1)
    if z is None:
        return dd, torch.zeros_like(dd)
    z = R.f64(z)
    return dd * R.act(act, z)[1], dd.abs() * R.act_error(z)


def check_grad(dd, a, b, z, act, gated, got, dtype):
    dz, e = grad_want(dd, z, act, gated)
    half = R.HALF[T[dtype]] if z is not None else 0.0
    e1 = e * (1 + 2.0 ** -7) + half * dz.abs() * (1 + 2.0 ** -7) + (R.TINY[T[dtype]] if z is not None else 0.0)
    A, B = R.f64(a), R.f64(b)
    R.close(got[0], dz @ B, e1 @ B.abs() + R.sum_error(dz.abs() @ B.abs(), dz.shape[1]), T[dtype])
    R.close(got[1], dz.T @ A, e1.T @ A.abs() + R.sum_error(dz.abs().T @ A.abs(), dz.shape[0]), T[dtype])
    if len(got) > 2:
        R.close(got[2], dz.sum(0), e.sum(0) + (dz.shape[0] + 8) * 2.0 ** -24 * dz.abs().sum(0) + 2.0 ** -23 * dz.abs().sum(0),
                torch.float32)


GRAD_SHAPES = [(1, 8, 8), (1, 256, 512), (5, 33, 70), (64, 128, 192), (65, 136, 72), (128, 512, 256), (200, 257, 129),
               (333, 640, 520), (1000, 128, 64), (513, 96, 1000)]


@pytest.mark.parametrize("m, n, k", GRAD_SHAPES)
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_matmul_grad(dtype, m, n, k):
    for i, (bias, act) in enumerate([(False, None), (True, None), (True, "gelu"), (False, "relu"), (True, "silu")]):
        say("matmul_grad", dtype, m, n, k, bias, act)
        g = gen(m + n + k + i)
        dd, a, b = normal(g, (m, n), dtype, 0.5), normal(g, (m, k), dtype), normal(g, (n, k), dtype, k ** -0.5)
        z = normal(g, (m, n), dtype) if act else None
        got = H.MatmulGrad(m, n, k, dtype, bias=bias, activation=act)(*([dd, a, b] + ([z] if act else [])))
        check_grad(dd, a, b, z, act, False, got, dtype)


@pytest.mark.parametrize("strides", [{"dd": 136, "a": 80, "b": 88, "z": 144, "da": 72, "db": 96},
                                     {"dd": 129, "a": 75, "b": 77, "z": 131, "da": 73, "db": 81}])
@pytest.mark.parametrize("act", [None, "silu"])
def test_matmul_grad_row_strides(act, strides):
    m, n, k = 150, 128, 72
    strides = {name: v for name, v in strides.items() if act or name != "z"}
    g = gen(m)
    dd, a, b = (normal(g, s, "bf16", 0.3, strides[x]) for x, s in (("dd", (m, n)), ("a", (m, k)), ("b", (n, k))))
    z = normal(g, (m, n), "bf16", 1.0, strides["z"]) if act else None
    got = H.MatmulGrad(m, n, k, "bf16", activation=act, bias=True, strides=strides)(*([dd, a, b] + ([z] if act else [])))
    check_grad(dd, a, b, z, act, False, got, "bf16")


def test_matmul_grad_large_tiles():
    m, n, k = 2304, 2200, 2120
    g = gen(m)
    dd, a, b = normal(g, (m, n), "bf16", 0.1), normal(g, (m, k), "bf16"), normal(g, (n, k), "bf16", 0.02)
    check_grad(dd, a, b, None, None, False, H.MatmulGrad(m, n, k, "bf16")(dd, a, b), "bf16")


@pytest.mark.parametrize("m, n, k", [(1, 16, 64), (1, 1408, 512), (5, 40, 200), (16, 33, 96), (24, 512, 1024),
                                     (40, 64, 512), (65, 64, 128), (130, 200, 264), (257, 129, 1000), (600, 1024, 512),
                                     (2100, 1152, 128), (3, 7, 5)])
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f8e4m3", "s8"])
def test_gated(dtype, m, n, k):
    for i, (act, save, out) in enumerate([("silu", False, "bf16"), ("gelu", True, "f32"), ("relu", True, "f16")]):
        say("gated", dtype, m, n, k, act, save, out)
        g = gen(m + 3 * n + k + i)
        ops = operands(g, m, 2 * n, k, dtype)
        got = H.GatedFeedForward(m, n, k, dtype, out_dtype=out, activation=act, save=save)(*ops)
        z, mag = sums(ops)
        err = R.sum_error(mag, k) + 4 * 2.0 ** -24 * mag
        if save:
            R.close(got[1], z, err, T[out])
            got = got[0]
        f = R.act(act, z[:, :n])[0]
        f_err = 1.2 * err[:, :n] + (R.act_error(z[:, :n]) if act != "relu" else 0)
        u, u_err = z[:, n:], err[:, n:]
        R.close(got, f * u, f_err * (u.abs() + u_err) + f.abs() * u_err + (f * u).abs() * 2.0 ** -24, T[out])


@pytest.mark.parametrize("m, n, k", [(1, 8, 8), (5, 33, 70), (64, 128, 192), (200, 257, 129), (333, 320, 520)])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_gated_grad(dtype, m, n, k):
    for act in ("silu", "gelu", "relu"):
        say("gated_grad", dtype, m, n, k, act)
        g = gen(m + n + k)
        dd, a, b = normal(g, (m, n), dtype, 0.5), normal(g, (m, k), dtype), normal(g, (2 * n, k), dtype, k ** -0.5)
        z = normal(g, (m, 2 * n), dtype)
        check_grad(dd, a, b, z, act, True, H.GatedFeedForwardGrad(m, n, k, dtype, activation=act)(dd, a, b, z), dtype)


# --------------------------------------------------------------------------
# gradients against differences
# --------------------------------------------------------------------------
def difference(f, tensors, directions, step=1e-5):
    """The central difference of sum(f) in 64 bits along each direction."""
    out = []
    for i, v in enumerate(directions):
        ends = []
        for s in (step, -step):
            at = list(tensors)
            at[i] = at[i] + s * v
            ends.append(f(*at).sum())
        out.append(float(ends[0] - ends[1]) / (2 * step))
    return out


@pytest.mark.parametrize("act", [None, "gelu", "silu"])
def test_matmul_grad_against_differences(act):
    m, n, k = 20, 24, 32
    g = gen(5)
    dd, a, b, bias = (normal(g, s, "bf16") for s in ((m, n), (m, k), (n, k), (n,)))
    z = (R.f64(a) @ R.f64(b).T + R.f64(bias))
    zt = z.to(torch.bfloat16).cuda()
    got = H.MatmulGrad(m, n, k, "bf16", bias=True, activation=act)(*([dd, a, b] + ([zt] if act else [])))
    v = [torch.randn(s, generator=g, dtype=torch.float64) for s in ((m, k), (n, k), (n,))]
    want = difference(lambda a, b, c: R.f64(dd) * R.act(act, a @ b.T + c)[0], [R.f64(a), R.f64(b), R.f64(bias)], v)
    # z is kept in bf16, so act' is taken up to 2^-8 |z| away (its slope is at
    # most 1.2), and dz and the results are rounded: three half steps in all
    mag = (R.f64(dd).abs() * (1.2 + 1.2 * z.abs()))
    bounds = [(mag @ R.f64(b).abs() * v[0].abs()).sum(), (mag.T @ R.f64(a).abs() * v[1].abs()).sum(),
              (mag.sum(0) * v[2].abs()).sum()]
    for t, w, d, e in zip(got, want, v, bounds):
        assert abs(float((R.f64(t) * d).sum()) - w) <= 3 * 2.0 ** -8 * float(e)


def test_gated_grad_against_differences():
    m, n, k = 12, 16, 32
    g = gen(6)
    dd, a, b = normal(g, (m, n), "f16"), normal(g, (m, k), "f16"), normal(g, (2 * n, k), "f16", 0.3)
    z = R.f64(a) @ R.f64(b).T
    got = H.GatedFeedForwardGrad(m, n, k, "f16")(dd, a, b, z.to(torch.float16).cuda())
    v = [torch.randn(s, generator=g, dtype=torch.float64) for s in ((m, k), (2 * n, k))]

    def f(a, b):
        z = a @ b.T
        return R.f64(dd) * R.act("silu", z[:, :n])[0] * z[:, n:]
    want = difference(f, [R.f64(a), R.f64(b)], v)
    gate, up = z[:, :n].abs(), z[:, n:].abs()
    mag = torch.cat([R.f64(dd).abs() * up * (1.2 + gate), R.f64(dd).abs() * (1 + 2 * gate)], 1)
    bounds = [(mag @ R.f64(b).abs() * v[0].abs()).sum(), (mag.T @ R.f64(a).abs() * v[1].abs()).sum()]
    for t, w, d, e in zip(got, want, v, bounds):
        assert abs(float((R.f64(t) * d).sum()) - w) <= 3 * 2.0 ** -11 * float(e)


def test_norm_grad_against_differences():
    rows, cols = 6, 100
    g = gen(8)
    dy, x, w = normal(g, (rows, cols), "f32"), normal(g, (rows, cols), "f32"), normal(g, (cols,), "f32")
    _, rstd = H.RmsNorm(rows, cols, "f32", eps=1e-3)(x, w)
    dx, dw = H.RmsNormGrad(rows, cols, "f32")(dy, x, w, rstd)
    v = [torch.randn(s, generator=g, dtype=torch.float64) for s in ((rows, cols), (cols,))]

    def f(x, w):
        return R.f64(dy) * x * (x.square().mean(1, keepdim=True) + 1e-3).rsqrt() * w
    want = difference(f, [R.f64(x), R.f64(w)], v)
    # about a hundred 32-bit roundings of terms whose sum of magnitudes is:
    mags = [(R.f64(dx).abs() * v[0].abs()).sum() + (R.f64(dy) * R.f64(w) * v[0]).abs().sum(),
            (R.f64(dy).abs() * R.f64(x).abs() @ v[1].abs()).sum()]
    for t, want_, d, e in zip((dx, dw), want, v, mags):
        assert abs(float((R.f64(t) * d).sum()) - want_) <= 200 * 2.0 ** -24 * float(e)


# --------------------------------------------------------------------------
# dropout
# --------------------------------------------------------------------------
def state(seed, offset):
    return torch.tensor([seed, offset], dtype=torch.int64, device="cuda")


@pytest.mark.parametrize("rows, cols, stride", [(1, 1, None), (1, 7, None), (3, 8, None), (5, 1001, None),
                                                (64, 4096, None), (9, 64, 72), (9, 61, 64), (7, 33, 35), (2, 100000, None)])
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
def test_dropout(dtype, rows, cols, stride):
    for p, res, seed, offset in ((0.1, True, 1234567890123456789, 2 ** 32 - 3), (0.5, False, -5, 2 ** 63 - 1),
                                 (0.0, True, 0, 0), (0.99999, False, 7, -1)):
        say("dropout", dtype, rows, cols, stride, p)
        g = gen(rows + cols)
        x = normal(g, (rows, cols), dtype, stride=stride)
        r = normal(g, (rows, cols), dtype, 2.0, stride) if res else None
        strides = {} if stride is None else {"x": stride, "y": stride + 8} | ({"residual": stride} if res else {})
        op = H.Dropout(rows, cols, dtype, p=p, residual=res, strides=strides)
        y = op(*([x, state(seed, offset)] + ([r] if res else [])))
        cut = round(p * 65536)
        if cut == 65536:
            keep, scale = torch.zeros(rows * cols, dtype=torch.bool), 0.0
        else:
            keep, scale = R.keep_mask(rows * cols, seed, offset, p)
        want = torch.where(keep.reshape(rows, cols), R.f64(x) * scale, 0.0)
        err = want.abs() * 2.0 ** -23
        if res:
            want = want + R.f64(r)
            err = err + want.abs() * 2.0 ** -24
        R.close(y, want, err, T[dtype])
        if not res:
            assert torch.equal(y.cpu() != 0, keep.reshape(rows, cols) & (x.cpu() != 0))


def test_dropout_backward_has_the_same_mask_and_drops_nan():
    """The gradient operator keeps what the forward pass kept, whatever the
    values are: a dropped NaN or infinity is 0."""
    rows, cols = 33, 257
    g = gen(3)
    s = state(99, 1000)
    x = normal(g, (rows, cols), "f32").abs() + 1
    y = H.Dropout(rows, cols, "f32", p=0.3)(x, s)
    dy = torch.full((rows, cols), float("nan"), device="cuda")
    dx = H.Dropout(rows, cols, "f32", p=0.3)(dy, s)
    assert torch.equal(torch.isnan(dx), y != 0) and (dx[y == 0] == 0).all()


def test_dropout_share():
    """The kept share of 2^24 elements lies within 6 standard deviations."""
    n, p = 1 << 24, 0.1
    y = H.Dropout(4096, 4096, "f16", p=p)(torch.ones((4096, 4096), dtype=torch.float16, device="cuda"), state(42, 0))
    q = 1 - round(p * 65536) / 65536
    kept = int((y != 0).sum())
    assert abs(kept - n * q) < 6 * math.sqrt(n * q * (1 - q))


# --------------------------------------------------------------------------
# long arrays, streams, graphs, refusals at launch
# --------------------------------------------------------------------------
def test_offsets_past_32_bits():
    """Arrays of more than 2^31 elements: the last rows are right."""
    rows, cols = 540000, 4096
    x = torch.empty((rows, cols), dtype=torch.bfloat16, device="cuda").fill_(0.5)
    g = gen(1)
    tail = (torch.randn((4, cols), generator=g)).to(torch.bfloat16)
    x[-4:] = tail.cuda()
    w = normal(g, (cols,), "bf16")
    say("norm past 2^31")
    y, rstd = H.RmsNorm(rows, cols, "bf16")(x, w)
    check_norm(x[-4:], w, None, "bf16", 1e-5, [y[-4:], rstd[-4:]])
    say("dropout past 2^31")
    del y
    y = H.Dropout(rows, cols, "bf16", p=0.25)(x, state(5, 6))
    keep, scale = R.keep_mask(4 * cols, 5, 6, 0.25, first=(rows - 4) * cols)
    want = torch.where(keep.reshape(4, cols), R.f64(tail) * scale, 0.0)
    R.close(y[-4:], want, want.abs() * 2.0 ** -23, torch.bfloat16)
    del y
    say("matmul past 2^31")
    b = normal(g, (64, cols), "bf16", 0.1)
    d = H.Matmul(rows, 64, cols, "bf16", out_dtype="f32")(x, b)
    check_matmul([x[-300:], b], {}, d[-300:], "f32", None, False)
    say("matmul_grad past 2^31")
    dd = torch.zeros((rows, 64), dtype=torch.bfloat16, device="cuda")
    dd[-300:] = normal(g, (300, 64), "bf16")
    da, db = H.MatmulGrad(rows, 64, cols, "bf16")(dd, x, b)
    check_grad(dd[-300:], x[-300:], b, None, None, False, [da[-300:], db], "bf16")


def layer_ops(m, h, f):
    """A feed-forward layer, forward and backward, as bound launches."""
    g = gen(m)
    x, r = normal(g, (m, h), "bf16"), normal(g, (m, h), "bf16")
    wn, wg, wd = normal(g, (h,), "bf16"), normal(g, (2 * f, h), "bf16", h ** -0.5), normal(g, (h, f), "bf16", f ** -0.5)
    s, dout = state(3, 4), normal(g, (m, h), "bf16")
    norm = H.RmsNorm(m, h, "bf16", residual=True).bind(x, wn, r)
    y, stream, rstd = norm.results
    gate = H.GatedFeedForward(m, f, h, "bf16", save=True).bind(y, wg)
    act, z = gate.results
    down = H.Matmul(m, h, f, "bf16").bind(act, wd)
    drop = H.Dropout(m, h, "bf16", p=0.1, residual=True).bind(down.results, s, stream)
    ddrop = H.Dropout(m, h, "bf16", p=0.1).bind(dout, s)
    ddown = H.MatmulGrad(m, h, f, "bf16").bind(ddrop.results, act, wd)
    dact, dwd = ddown.results
    dgate = H.GatedFeedForwardGrad(m, f, h, "bf16").bind(dact, y, wg, z)
    dy, dwg = dgate.results
    dnorm = H.RmsNormGrad(m, h, "bf16", stream_grad=True).bind(dy, stream, wn, rstd, dout)
    chain = [norm, gate, down, drop, ddrop, ddown, dgate, dnorm]
    return chain, x, s, [drop.results, dwd, dwg, *dnorm.results]


@pytest.mark.parametrize("m", [3, 100, 700])
def test_graph_replays_equal_eager(m):
    """The whole layer captured: replays with other inputs and another state,
    with eager work between them, equal the eager results bit for bit."""
    chain, x, s, results = layer_ops(m, 512, 768)
    for c in chain:
        c()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for c in chain:
            c()
    g = gen(9)
    for turn in range(4):
        x.copy_(torch.randn(x.shape, generator=g).to(torch.bfloat16))
        s.add_(1000)
        for c in chain:
            c()
        want = [t.clone() for t in results]
        for t in results:
            t.zero_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for k, (t, w) in enumerate(zip(results, want)):
            assert torch.equal(t, w), (turn, k)


def test_other_streams_and_noalloc():
    """One handle on two streams at once, each with its own buffers; the
    no-allocation launch equals the ordinary one."""
    m, n, k = 100, 256, 4096
    op = H.Matmul(m, n, k, "bf16", out_dtype="f32")
    assert op.workspace_bytes > 0
    sets = [operands(gen(i), m, n, k, "bf16") for i in range(2)]
    want = [op(*o).clone() for o in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    launches = [op.bind(*o, stream=st) for o, st in zip(sets, streams)]
    for _ in range(20):
        for launch, st in zip(launches, streams):
            launch(st)
    torch.cuda.synchronize()
    for launch, w in zip(launches, want):
        assert torch.equal(launch.results, w)
    out = torch.empty_like(want[0])
    op.launch_noalloc_ptrs([t.data_ptr() for t in sets[0]], [out.data_ptr()], torch.cuda.current_stream().cuda_stream)
    torch.cuda.synchronize()
    assert torch.equal(out, want[0])
    big = H.MatmulGrad(4096, 4096, 64, "bf16", activation="relu")
    assert big.workspace_bytes > H.SCRATCH_BYTES
    z = torch.zeros((4096, 4096), dtype=torch.bfloat16, device="cuda")
    small = torch.zeros((4096, 64), dtype=torch.bfloat16, device="cuda")
    outs = [torch.empty_like(small) for _ in range(2)]
    with pytest.raises(H.FusionError) as e:
        big.launch_noalloc_ptrs([t.data_ptr() for t in (z, small, small, z.clone())], [t.data_ptr() for t in outs])
    assert e.value.status == "HF_ERR_UNSUPPORTED"


def test_launch_refusals():
    op = H.Matmul(4, 32, 64, "bf16")
    a, b = torch.zeros((4, 64), dtype=torch.bfloat16, device="cuda"), torch.zeros((32, 64), dtype=torch.bfloat16, device="cuda")
    d = torch.zeros((4, 32), dtype=torch.bfloat16, device="cuda")
    A, B, D = a.data_ptr(), b.data_ptr(), d.data_ptr()
    host = torch.zeros((4, 64), dtype=torch.bfloat16).pin_memory()

    def refused(params, results, text, status="HF_ERR_INVALID", op=op, ws=0):
        with pytest.raises(H.FusionError) as e:
            op.launch_ptrs(params, results, 0, ws)
        assert e.value.status == status and text in e.value.message, e.value.message
    refused([A], [D], "expected 2 parameter")
    refused([A, B], [D, D], "expected 2 parameter")
    refused([0, B], [D], "a must be a non-NULL")
    refused([A + 2, B], [D], "16-byte aligned")
    refused([host.data_ptr(), B], [D], "device memory")
    refused([A, B], [A], "overlaps a")
    refused([A, B + 16], [B], "overlaps b")
    # an extent that runs past its allocation
    whole = torch.empty(64 << 20, dtype=torch.uint8, device="cuda")
    # (torch may have cut the tensor from a larger one: its allocation's end)
    end = [g["address"] + g["total_size"] for g in torch.cuda.memory_snapshot()
           if g["address"] <= whole.data_ptr() < g["address"] + g["total_size"]][0]
    refused([end - 16, B], [D], "past the end")
    split = H.Matmul(100, 256, 4096, "bf16")
    assert split.workspace_bytes > 0
    x, y = torch.zeros((100, 4096), dtype=torch.bfloat16, device="cuda"), torch.zeros((256, 4096), dtype=torch.bfloat16, device="cuda")
    z = torch.zeros((100, 256), dtype=torch.bfloat16, device="cuda")
    ptrs = [x.data_ptr(), y.data_ptr()]
    refused(ptrs, [z.data_ptr()], "needs a workspace", op=split)
    refused(ptrs, [z.data_ptr()], "overlaps", op=split, ws=y.data_ptr())
    with pytest.raises(ValueError, match="a must be a GPU tensor"):
        op(a.float(), b)
    with pytest.raises(ValueError, match="b must be a GPU tensor"):
        op(a, b.cpu())
    with pytest.raises(ValueError, match="a must be a GPU tensor"):
        op(torch.zeros((4, 128), dtype=torch.bfloat16, device="cuda")[:, ::2], b)
    with pytest.raises(ValueError, match="expected 2 parameters"):
        op(a)
    with pytest.raises(ValueError, match="expected 1 results"):
        op(a, b, out=[d, d])
    with pytest.raises(ValueError, match="workspace"):
        split(x, y, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
    torch.cuda.synchronize()


def test_column_windows_of_one_array():
    """A result beside its parameter in the same rows is no overlap."""
    base = torch.randn((40, 256), generator=gen(2)).to(torch.bfloat16).cuda()
    w = torch.ones(128, dtype=torch.bfloat16, device="cuda")
    op = H.RmsNorm(40, 128, "bf16", strides={"x": 256, "y": 256})
    rstd = torch.empty(40, device="cuda")
    x = base[:, :128].clone()
    op(base[:, :128], w, out=[base[:, 128:], rstd])
    check_norm(x, w, None, "bf16", 1e-5, [base[:, 128:], rstd])
    assert torch.equal(base[:, :128], x)
    with pytest.raises(H.FusionError):
        op(base[:, :128], w, out=[base[:, 64:192], rstd])


@pytest.mark.parametrize("m, n, k", [(2050, 4096, 512), (4099, 2048, 640), (4160, 2080, 264)])
def test_matmul_last_rows(m, n, k):
    """A few rows past whole tiles, which may be a strip of their own: every
    operand and result of theirs lies at an offset."""
    for dtype, out, act in (("bf16", "bf16", "silu"), ("f8e4m3", "f16", None)):
        say("matmul", dtype, m, n, k)
        g = gen(m + k)
        ops = operands(g, m, n, k, dtype)
        extra = {"bias": normal(g, (n,), out), "residual": normal(g, (m, n), out, stride=n + 16)}
        op = H.Matmul(m, n, k, dtype, out_dtype=out, bias=True, activation=act, residual=True, save=True,
                      strides={"residual": n + 16, "z": n + 8})
        check_matmul(ops, extra, op(*ops, *extra.values()), out, act, True)


def test_gated_last_rows():
    m, n, k = 2060, 2048, 320
    g = gen(m)
    ops = operands(g, m, 2 * n, k, "s8")
    d, zs = H.GatedFeedForward(m, n, k, "s8", out_dtype="f16", activation="relu", save=True)(*ops)
    z, mag = sums(ops)
    err = R.sum_error(mag, k) + 4 * 2.0 ** -24 * mag
    R.close(zs, z, err, torch.float16)
    f, u = R.act("relu", z[:, :n])[0], z[:, n:]
    R.close(d, f * u, err[:, :n] * (u.abs() + err[:, n:]) + f.abs() * err[:, n:] + (f * u).abs() * 2.0 ** -24, torch.float16)


@pytest.mark.parametrize("m, n, k", [(1, 8500, 384), (7, 8400, 1000), (33, 8330, 72), (64, 20000, 264), (9, 40, 4096)])
def test_strips(m, n, k):
    """Many columns take strips from one row on; more strips than compute
    units; a few columns shared by many workgroups."""
    for dtype, out in (("bf16", "bf16"), ("s8", "f32"), ("f8e4m3", "f16")):
        say("strips", dtype, m, n, k, H.Matmul(m, n, k, dtype, out_dtype=out, mode="plan").plan())
        g = gen(m + n)
        ops = operands(g, m, n, k, dtype)
        extra = {"bias": normal(g, (n,), out)}
        op = H.Matmul(m, n, k, dtype, out_dtype=out, bias=True, activation="relu")
        check_matmul(ops, extra, op(*ops, *extra.values()), out, "relu", False)
    gops = operands(gen(m), m, 2 * (n // 2), k, "f16")
    z, mag = sums(gops)
    err, half = R.sum_error(mag, k) + 4 * 2.0 ** -24 * mag, n // 2
    d = H.GatedFeedForward(m, half, k, "f16", out_dtype="f32", activation="relu")(*gops)
    f, u = R.act("relu", z[:, :half])[0], z[:, half:]
    R.close(d, f * u, err[:, :half] * (u.abs() + err[:, half:]) + f.abs() * err[:, half:] + (f * u).abs() * 2.0 ** -24,
            torch.float32)
