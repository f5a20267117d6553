"""examples/expert_layer.py: the training step's gradients against autograd in
64 bits, replays of its graph, and the served layer against the trained one."""
import os
import sys

import pytest
import torch

import operators_reference as R

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
import expert_layer as E  # noqa: E402

pytestmark = pytest.mark.gpu


def made(tokens, top_k, experts, hidden, inner, dtype, seed=3):
    l = E.TrainingStep(tokens, top_k, experts, hidden, inner, dtype, seed)
    g = torch.Generator(device="cuda").manual_seed(seed)
    l.x.copy_(torch.randn(l.x.shape, generator=g, device="cuda"))
    l.target.copy_(torch.randn(l.x.shape, generator=g, device="cuda"))
    l.route(torch.randn((tokens, experts), generator=g, device="cuda"))
    return l


def wanted(l, experts, inner):
    """y and the gradients in x, the choices' weights, gate_up and down."""
    x, share, up, down = (R.f64(t).requires_grad_() for t in (l.x, l.share, l.weight["gate_up"], l.weight["down"]))
    hidden, rows = x.shape[1], []
    for t in range(x.shape[0]):
        y = x[t]
        for j in range(share.shape[1]):
            e = int(l.expert[t, j])
            z = up[e * 2 * inner:(e + 1) * 2 * inner] @ x[t]
            y = y + share[t, j] * (down[e * hidden:(e + 1) * hidden] @ (torch.nn.functional.silu(z[:inner]) * z[inner:]))
        rows.append(y)
    y = torch.stack(rows)
    (0.5 * (y - R.f64(l.target)).square().sum() / x.shape[0]).backward()
    return [y.detach(), x.grad, share.grad, up.grad, down.grad]


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("tokens, top_k, experts, hidden, inner", [(33, 2, 4, 64, 48), (20, 3, 7, 72, 40), (1, 2, 9, 128, 24)])
def test_gradients(dtype, tokens, top_k, experts, hidden, inner):
    l = made(tokens, top_k, experts, hidden, inner, dtype)
    l.forward(), l.backward()
    # nine arrays on the longest way are rounded to dtype, one after another
    bound = 9 * R.HALF[l.x.dtype]
    for k, (got, want) in enumerate(zip([l.y, l.dx, l.grad_share, l.grad_gate_up, l.grad_down], wanted(l, experts, inner))):
        off = float((R.f64(got) - want).norm() / want.norm())
        assert off < bound, (k, off)


def test_steps_replay_what_eager_calls_give():
    a, b = (made(200, 2, 6, 128, 96, "bf16") for _ in range(2))
    for i in range(3):
        a.step(lr=0.5)
        b.forward(), b.backward()
        for name, grad in (("gate_up", b.grad_gate_up), ("down", b.grad_down)):
            b.master[name].sub_(grad.float(), alpha=0.5)
            b.weight[name].copy_(b.master[name])
        # new choices between the replays
        g = torch.Generator(device="cuda").manual_seed(i)
        scores = torch.randn((200, 6), generator=g, device="cuda")
        a.route(scores), b.route(scores)
        torch.cuda.synchronize()
        for name in a.master:
            assert torch.equal(a.master[name], b.master[name]), (i, name)


@pytest.mark.parametrize("tokens", [1, 5, 300])
def test_served(tokens):
    experts, hidden, inner = 5, 256, 200
    l = made(tokens, 2, experts, hidden, inner, "bf16")
    l.forward()
    y = E.Served(l.master, experts)(l.x, l.expert, l.share)
    # weights and rows in e4m3: values of a block are off by 2^-5 of themselves
    # in the mean square at most (half a step of 2^-3 at the most), in three
    # factors of a term, whose errors are independent; twice that is the bound
    diff = R.f64(y) - R.f64(l.y)
    added = R.f64(l.y) - R.f64(l.x)
    assert float(diff.norm() / added.norm()) < 2 * 3 ** 0.5 * 2.0 ** -4


def test_runs(capsys):
    E.main()
    out = capsys.readouterr().out
    assert out.count("step") == 5 and out.count("served") == 3
