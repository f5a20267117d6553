"""Launches of more workgroups than a grid's first dimension holds (2^32
threads), and arrays of tens of gigabytes: the sizes that the header promises."""
import pytest
import torch

import compiler_hlo_amd as H
import operators_reference as R

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def room():
    torch.cuda.empty_cache()
    yield
    torch.cuda.empty_cache()


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


@pytest.mark.parametrize("rows, cols", [((1 << 26) + 5, 8), ((1 << 24) + 3, 1032)])
def test_norm_rows(rows, cols):
    """A workgroup for 4 short rows, or one for each: over 2^32 threads."""
    g = gen(rows)
    x = torch.empty((rows, cols), dtype=torch.bfloat16, device="cuda").normal_(generator=g)
    w = torch.empty(cols, dtype=torch.bfloat16, device="cuda").normal_(generator=g)
    y, rstd = H.RmsNorm(rows, cols, "bf16")(x, w)
    print("norm", rows, cols, flush=True)
    for at in [0, 1 << 20, rows // 2, rows - 4000]:
        s = x[at:at + 4000].double()
        want = (s.square().mean(1) + 1e-5).rsqrt()
        # the mean, its root and two products: rows of up to 1032 add with 70 roundings
        R.close(rstd[at:at + 4000], want.cpu(), want.cpu() * 80 * 2.0 ** -24, torch.float32)
        want = (s * want[:, None] * w.double()).cpu()
        R.close(y[at:at + 4000], want, want.abs() * 80 * 2.0 ** -24, torch.bfloat16)
    # every row has been written
    step = 1 << 22
    for at in range(0, rows, step):
        s = x[at:at + step].float()
        r = (s.square().mean(1) + 1e-5).rsqrt()
        assert ((rstd[at:at + step] - r).abs() <= 160 * 2.0 ** -24 * r).all()


def test_dropout_of_more_than_2_35_elements():
    rows, cols = (1 << 22) + 1, 8192
    x = torch.empty((rows, cols), dtype=torch.bfloat16, device="cuda").fill_(0.5)
    x[-1] = torch.empty(cols, dtype=torch.bfloat16, device="cuda").normal_(generator=gen(2))
    s = torch.tensor([5, 6], dtype=torch.int64, device="cuda")
    y = H.Dropout(rows, cols, "bf16", p=0.25)(x, s)
    print("dropout", rows, cols, flush=True)
    for row in (0, rows // 2, rows - 2, rows - 1):
        keep, scale = R.keep_mask(cols, 5, 6, 0.25, first=row * cols)
        want = torch.where(keep, R.f64(x[row]) * scale, 0.0)
        R.close(y[row], want, want.abs() * 2.0 ** -23, torch.bfloat16)


def test_norm_gradient_of_one_far_row():
    """The fold of 2^26 columns and a few."""
    cols = (1 << 26) + 24
    g = gen(3)
    dy, h = (torch.empty((1, cols), dtype=torch.bfloat16, device="cuda").normal_(generator=g) for _ in range(2))
    w = torch.ones(cols, dtype=torch.bfloat16, device="cuda")
    rstd = torch.ones(1, device="cuda")
    dx, dw = H.RmsNormGrad(1, cols, "bf16")(dy, h, w, rstd)
    print("norm_grad", cols, flush=True)
    assert torch.equal(dw, dy[0].float() * h[0].float())  # exact in 32 bits
    assert torch.isfinite(dx).all()


def test_strips_of_2_30_columns():
    """No contraction: the result is the bias."""
    n = 1 << 30
    bias = torch.empty(n, dtype=torch.bfloat16, device="cuda").normal_(generator=gen(4))
    half = dict(dtype=torch.bfloat16, device="cuda")
    d = H.Matmul(1, n, 0, bias=True)(torch.empty((1, 0), **half), torch.empty((n, 0), **half), bias)
    print("strips", n, flush=True)
    assert torch.equal(d[0], bias)
