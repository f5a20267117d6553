"""examples/feed_forward.py: the layer's values and gradients against a plain
64-bit form, its training under a graph, and its 8-bit serving."""
import os
import sys

import pytest
import torch

import operators_reference as R

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

pytestmark = pytest.mark.gpu


def relative(got, want):
    return float((R.f64(got) - want).norm() / want.norm())


def test_layer_against_autograd_in_64_bits():
    """Without dropout.  Each tensor between the operators is rounded to bf16
    (2^-9 of its norm, a random rounding's size); six of them lie on the
    longest path."""
    import feed_forward as F
    rows, hidden, inner = 200, 256, 384
    layer = F.TrainingStep(rows, hidden, inner, p=0.0)
    g = torch.Generator(device="cuda").manual_seed(2)
    layer.x.copy_(torch.randn(layer.x.shape, generator=g, device="cuda"))
    layer.target.copy_(torch.randn(layer.x.shape, generator=g, device="cuda"))
    layer.forward(), layer.backward()
    x, wn, wg, wd = (R.f64(t).requires_grad_() for t in (layer.x, *layer.weight.values()))
    h = x * (x.square().mean(1, keepdim=True) + 1e-5).rsqrt() * wn
    z = h @ wg.T
    y = x + (torch.nn.functional.silu(z[:, :inner]) * z[:, inner:]) @ wd.T
    (0.5 * (y - R.f64(layer.target)).square().sum() / rows).backward()
    assert relative(layer.y, y.detach()) < 6 * 2.0 ** -9
    for got, want in ((layer.dx, x), (layer.grad_norm, wn), (layer.grad_gate_up, wg), (layer.grad_down, wd)):
        assert relative(got, want.grad) < 6 * 2.0 ** -9


def test_training_lowers_the_loss_and_serving_agrees():
    import feed_forward as F
    layer = F.TrainingStep(300, 256, 512, p=0.1)
    g = torch.Generator(device="cuda").manual_seed(3)
    layer.x.copy_(torch.randn(layer.x.shape, generator=g, device="cuda"))
    layer.target.copy_(layer.x.roll(1, 1))
    layer.step(0.05)
    first = layer.loss()
    for _ in range(40):
        layer.step(0.05)
    assert layer.loss() < 0.9 * first
    for kind, step in (("f8e4m3", 2.0 ** -4), ("s8", 4.0 / 127)):
        served = F.Served(layer.master, kind)
        for rows in (1, 20, 300):
            x = layer.x[:rows].contiguous()
            y, stream = served(x, torch.zeros_like(x))
            assert torch.equal(stream, x)
            w = {k: R.f64(v) for k, v in layer.master.items()}
            v = R.f64(x)
            h = v * (v.square().mean(1, keepdim=True) + 1e-5).rsqrt() * w["norm"]
            z = h @ w["gate_up"].T
            want = (torch.nn.functional.silu(z[:, :512]) * z[:, 512:]) @ w["down"].T
            # two operands quantised by at most half a step each, through a
            # product of two such sums
            assert relative(R.f64(y) - v, want) < 4 * step


def test_both_products_are_served_in_8_bits():
    """Rows and weights of both products in 8 bits.  Each of the four arrays is
    off by e of its norm: in e4m3 half a step of 2^-4, spread evenly, at most
    2^-4 / sqrt(3); in s8 a step of the row's largest value / 127 over
    sqrt(12), where that value is up to 4 times the root mean square of a normal row and 10
    times that of the gated product's.  Gate and up are then off by sqrt(2) e,
    their product by 1.43 of that (silu keeps a normal value's spread), and the
    down projection adds two more: 1.42 2^-4 in all for e4m3; for s8
    hypot(1.43 sqrt(2) 4, 4, 10) / (127 sqrt(12))."""
    import feed_forward as F
    g = torch.Generator(device="cuda").manual_seed(5)
    hidden, inner = 512, 1024
    make = lambda shape, s: torch.randn(shape, generator=g, device="cuda") * s  # noqa: E731
    master = {"norm": torch.ones(hidden, device="cuda"), "gate_up": make((2 * inner, hidden), hidden ** -0.5),
              "down": make((hidden, inner), inner ** -0.5)}
    for kind, bound in (("f8e4m3", 0.1), ("s8", 0.035)):
        served = F.Served(master, kind)
        for rows in (1, 9, 200):
            x = make((rows, hidden), 1.0).to(torch.bfloat16)
            y, _ = served(x, torch.zeros_like(x))
            products = [op for op in served.ops[rows] if not isinstance(op, F.H.RmsNorm)]
            assert len(products) == 2 and all(b.dtype == kind for op in products for b in op.params[:2])
            v = R.f64(x)
            h = v * (v.square().mean(1, keepdim=True) + 1e-5).rsqrt()
            z = h @ R.f64(master["gate_up"]).T
            want = (torch.nn.functional.silu(z[:, :inner]) * z[:, inner:]) @ R.f64(master["down"]).T
            # and the sum with the stream is rounded to bf16
            assert relative(R.f64(y) - v, want) < bound + 2.0 ** -8 * float((v + want).norm() / want.norm())


@pytest.mark.parametrize("kind", ["f8e4m3", "s8"])
def test_a_channel_of_zeros_is_served_as_zeros(kind):
    import feed_forward as F
    g = torch.Generator(device="cuda").manual_seed(6)
    master = {"norm": torch.ones(128, device="cuda"), "gate_up": torch.randn((512, 128), generator=g, device="cuda"),
              "down": torch.randn((128, 256), generator=g, device="cuda")}
    master["gate_up"][3] = 0.0
    master["down"][5] = 0.0
    x = torch.randn((4, 128), generator=g, device="cuda").to(torch.bfloat16)
    y, stream = F.Served(master, kind)(x, torch.zeros_like(x))
    assert torch.isfinite(y).all() and torch.equal(y[:, 5], stream[:, 5])
