"""The operators where 32 or 16 bits come to their ends: sums, scales,
activations, epsilons and gradients of unusual size."""
import math

import pytest
import torch

import compiler_hlo_amd as H
import operators_reference as R

pytestmark = pytest.mark.gpu


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


@pytest.mark.parametrize("m, n, k", [(1, 512, 100000), (8, 40, 131056), (5, 6000, 65600), (40, 512, 100000),
                                     (200, 300, 66000), (600, 4200, 2064)])
def test_s8_sums_are_exact(m, n, k):
    """Sums of s8 products are whole in 32 bits however the contraction is
    shared: large parts that cancel (or nearly reach 2^31) leave every unit."""
    g = gen(k)
    a = torch.randint(126, 128, (m, k), generator=g, device="cuda").to(torch.int8)
    b = torch.randint(120, 128, (n, k), generator=g, device="cuda").to(torch.int8)
    b[: n // 2, : k // 2] *= -1
    one = torch.ones(max(m, n), device="cuda")
    op = H.Matmul(m, n, k, "s8", out_dtype="f32")
    print("s8", m, n, k, op.plan(), flush=True)
    want = a.double() @ b.double().t()
    assert torch.equal(op(a, b, one[:m].contiguous(), one[:n].contiguous()), want.float())
    half = n // 2
    d, z = H.GatedFeedForward(m, half, k, "s8", out_dtype="f32", activation="relu", save=True)(
        a, b[: 2 * half], one[:m].contiguous(), one[: 2 * half].contiguous())
    assert torch.equal(z, want[:, : 2 * half].float())


@pytest.mark.parametrize("m", [1, 40, 200])
def test_scales_of_any_size(m):
    """z * a_scale * b_scale from the left: neither the two scales' product's
    overflow nor its loss of bits reaches a result that is in range."""
    n, k = 64, 1024
    a = torch.full((m, k), 127, dtype=torch.int8, device="cuda")
    b = torch.full((n, k), 127, dtype=torch.int8, device="cuda")
    b[: n // 2] = 0
    for sa, sb in ((1e-30, 3e-15), (1e25, 1e20), (1e25, 1e-30)):
        for make in (H.Matmul, H.GatedFeedForward):
            gated = make is H.GatedFeedForward
            sizes = (m, n // 2 if gated else n, k)
            d = make(*sizes, "s8", out_dtype="f32", **({"activation": "relu", "save": True} if gated else {}))(
                a, b, torch.full((m,), sa, device="cuda"), torch.full((n,), sb, device="cuda"))
            z = d[1] if gated else d
            assert (z[:, : n // 2] == 0).all()
            s = float(torch.tensor(sa)) * float(torch.tensor(sb)) * 127.0 * 127.0 * k
            want = torch.full((m, n // 2), s, dtype=torch.float64)
            # three roundings: the sum is whole
            R.close(z[:, n // 2:], want, want * 3 * 2.0 ** -24, torch.float32)


@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_activations_of_negative_values_in_32_bits(act):
    """Where z sigmoid(z) falls off exponentially, an f32 result keeps its
    relative precision: exp2 and the reciprocal (a unit each, of 2^-23), the
    argument's rest, 1 + exp and the product (half a unit each): 4 units and
    one to spare."""
    z = torch.cat([torch.linspace(-70, 0, 5000), torch.linspace(0, 60, 1000)]) if act == "silu" else \
        torch.cat([torch.linspace(-9, 0, 5000), torch.linspace(0, 9, 1000)])
    n = z.numel()
    one = torch.ones((n, 1), dtype=torch.bfloat16, device="cuda")
    d = H.Matmul(1, n, 1, "bf16", out_dtype="f32", bias=True, activation=act)(
        torch.zeros((1, 1), dtype=torch.bfloat16, device="cuda"), one, z.cuda())
    w = z.double()
    u = w if act == "silu" else 2 * math.sqrt(2 / math.pi) * (w + 0.044715 * w ** 3)
    want = w / (1 + torch.exp(-u))
    R.close(d[0], want, want.abs() * 5 * 2.0 ** -23, torch.float32)


def test_norm_epsilon_outside_32_bits():
    """Epsilon is a double: its root counts where it is in range itself."""
    x, w = torch.zeros((3, 40), device="cuda"), torch.ones(40, device="cuda")
    x[1] = 1e-24
    x[2] = 1.0
    for eps in (1e-50, 1e44):
        y, rstd = H.RmsNorm(3, 40, "f32", eps=eps)(x, w)
        want = (R.f64(x).square().mean(1) + eps).rsqrt()
        R.close(rstd, want, want * 16 * 2.0 ** -24, torch.float32)
        R.close(y, R.f64(x) * want[:, None], (R.f64(x) * want[:, None]).abs() * 18 * 2.0 ** -24, torch.float32)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_gradients_at_the_ends_of_their_range(dtype):
    """dz goes through the products in the operands' type: in f16 an infinity
    from 65520 on, which stays in its row of da and of db, and zero below
    2^-25.  dbias is summed before that rounding; bf16 keeps all of them."""
    m, n, k = 70, 40, 24
    g = gen(1)
    t = {"f16": torch.float16, "bf16": torch.bfloat16}[dtype]
    a, b = (torch.randint(1, 3, s, generator=g, device="cuda").to(t) for s in ((m, k), (n, k)))
    dd, z = torch.zeros((m, n), dtype=t, device="cuda"), torch.full((m, n), 1.5, dtype=t, device="cuda")
    dd[3, 7], dd[5, 8] = 61440.0, 2.0 ** -20
    z[3, 7], z[5, 8] = 2.5, -11.0
    slope = R.act("silu", torch.tensor([2.5, -11.0], dtype=torch.float64))[1].tolist()
    big, small = 61440.0 * slope[0], 2.0 ** -20 * slope[1]
    assert big > 65520 and abs(small) < 2.0 ** -25
    da, db, dbias = H.MatmulGrad(m, n, k, dtype, bias=True, activation="silu")(dd, a, b, z)
    rows, cols = torch.arange(m, device="cuda") == 3, torch.arange(n, device="cuda") == 7
    if dtype == "f16":
        assert (da[rows] == math.inf).all() and (db[cols] == math.inf).all()
        assert (da[~rows] == 0).all() and (db[~cols] == 0).all()
    else:
        half = 2.0 ** -8
        want = torch.zeros((m, k), dtype=torch.float64)
        want[3], want[5] = big * R.f64(b)[7], small * R.f64(b)[8]
        R.close(da, want, want.abs() * (half + 2.0 ** -14), t)
        want = torch.zeros((n, k), dtype=torch.float64)
        want[7], want[8] = big * R.f64(a)[3], small * R.f64(a)[5]
        R.close(db, want, want.abs() * (half + 2.0 ** -14), t)
    want = torch.zeros(n, dtype=torch.float64)
    want[7], want[8] = big, small
    R.close(dbias, want, want.abs() * 2.0 ** -14, torch.float32)
    # gated: the up half's value times the gradient
    half_n = n // 2
    zg = torch.ones((m, n), dtype=t, device="cuda")
    zg[:, half_n:] = 300.0
    dg = torch.zeros((m, half_n), dtype=t, device="cuda")
    dg[9, 2] = 300.0
    da, db = H.GatedFeedForwardGrad(m, half_n, k, dtype, activation="relu")(dg, a, b, zg)
    if dtype == "f16":
        assert (da[9] == math.inf).all() and (db[2] == math.inf).all()
    else:
        want = 90000.0 * R.f64(b)[2] + 300.0 * R.f64(b)[half_n + 2]
        R.close(da[9], want, want * 2 * half, t)
    others = torch.arange(m, device="cuda") != 9
    assert (da[others] == 0).all()
    assert torch.equal(db[half_n + 2], 300.0 * a[9])


def test_buffers_of_a_launch_on_another_stream_are_not_reused_before_it():
    """Tensors that the program drops right after a launch on a stream of its
    own: torch's allocator must not give their memory to the next tensor of
    the stream they came from while that launch is still waiting."""
    rows, cols = 64, 4096
    op = H.RmsNorm(rows, cols, "f32", residual=True)
    w = torch.ones(cols, device="cuda")
    x, r, y, h = (torch.full((rows, cols), v, device="cuda") for v in (1.0, 2.0, 0.0, 0.0))
    rstd = torch.empty(rows, device="cuda")
    taken = {t.data_ptr() for t in (x, r, y, h)}
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        torch.cuda._sleep(100_000_000)  # some 50 ms
    op(x, w, r, out=[y, h, rstd], stream=side)
    del x, r, y, h
    later = [torch.full((rows, cols), 9.0, device="cuda") for _ in range(4)]
    assert not taken & {t.data_ptr() for t in later}
    torch.cuda.synchronize()
    assert (rstd - (9.0 + 1e-5) ** -0.5).abs().max() < 1e-6


@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_activation_limits_in_32_bits(act):
    """f32 results at 0, far values, infinities and NaN."""
    inf, nan = math.inf, math.nan
    z = torch.tensor([0.0, 200.0, 1e30, 3e38, inf, -200.0, -1e30, -3e38, -inf, nan], device="cuda")
    one = torch.ones((10, 1), dtype=torch.bfloat16, device="cuda")
    d = H.Matmul(1, 10, 1, "bf16", out_dtype="f32", bias=True, activation=act)(one[:1] * 0, one, z)[0]
    assert torch.equal(d[:5], z[:5]) and (d[5:9] == 0).all() and torch.isnan(d[9])
