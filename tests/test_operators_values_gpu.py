"""The operators where 32 or 16 bits come to their ends: sums, scales,
activations, epsilons and gradients of unusual size."""
import pytest
import torch

import compiler_hlo_amd as H

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
