"""Operators by expert on arrays of more than 2^31 elements and sorts of many
pairs.  Values are small whole numbers, so every sum is exact."""
import pytest
import torch

import compiler_hlo_amd as H
import experts_reference as X
from test_operators_gpu import say

pytestmark = pytest.mark.gpu


def whole(shape, seed, top=2, dtype=torch.bfloat16):
    """Whole numbers of -top .. top, made in pieces."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    t = torch.empty(shape, dtype=dtype, device="cuda")
    for part in t.split(1 << 15):
        part.copy_(torch.randint(-top, top + 1, part.shape, generator=g, device="cuda"))
    return t


def test_sort_of_many_pairs():
    tokens, top_k, experts = 2_000_000, 8, 300
    g = torch.Generator().manual_seed(1)
    ids = torch.randint(-20, experts + 20, (tokens, top_k), generator=g, dtype=torch.int32)
    say("sort", tokens, top_k, experts)
    got = H.ExpertSort(tokens, top_k, experts)(ids.cuda())
    for a, b in zip(got, X.sort(ids, experts)):
        assert torch.equal(a.cpu(), b)


def test_rows_past_32_bits():
    """Dispatch, combine and its gradient with 2.3e9 elements by expert."""
    tokens, top_k, experts, cols = 70000, 8, 16, 4104
    pairs = tokens * top_k
    assert pairs * cols > 2 ** 31
    g = torch.Generator(device="cuda").manual_seed(2)
    ids = torch.randint(0, experts + 1, (tokens, top_k), generator=g, device="cuda", dtype=torch.int32)
    place, order, offsets = H.ExpertSort(tokens, top_k, experts)(ids)
    live = int(offsets[-1])
    x = whole((tokens, cols), 3)
    say("dispatch", pairs, cols)
    y = H.ExpertDispatch(tokens, top_k, cols)(x, place)
    token = (order // top_k).long()
    for r in (0, live // 2, 2 ** 31 // cols - 50, live - 100):
        assert torch.equal(y[r:r + 100], x[token[r:r + 100]])
    say("combine", pairs, cols)
    w = torch.randint(-2, 3, (tokens, top_k), generator=g, device="cuda").float()
    d = H.ExpertCombine(tokens, top_k, cols)(y, place, w)
    # all rows of a token are its own: d = x times the sum of its live weights
    total = torch.where(place >= 0, w, 0.0).sum(1, keepdim=True)
    for a, b, c in zip(d.split(8192), x.split(8192), total.split(8192)):
        assert torch.equal(a.float(), b.float() * c)
    say("combine gradient", pairs, cols)
    dy, dw = H.ExpertCombineGrad(tokens, top_k, cols)(x, y, place, w)
    for r in (0, 2 ** 31 // cols - 50, live - 100):
        o = order[r:r + 100].long()
        assert torch.equal(dy[r:r + 100].float(), w.reshape(-1)[o][:, None] * x[o // top_k].float())
    square = torch.cat([p.float().square().sum(1) for p in x.split(8192)])
    assert torch.equal(dw, torch.where(place >= 0, square[:, None], 0.0))


def test_products_past_32_bits():
    """A product by expert and its gradient over 2.2e9 elements of a."""
    m, n, k, experts = 540000, 72, 4096, 4
    assert m * k > 2 ** 31
    a, b, dd = whole((m, k), 4, 1), whole((experts * n, k), 5, 1), whole((m, n), 6, 1)
    ends = [0, 100000, 100001, 400000, 539990]
    offsets = torch.tensor(ends, dtype=torch.int32, device="cuda")
    say("product", m, n, k)
    d = H.Matmul(m, n, k, out_dtype="f32", experts=experts)(a, b, offsets)
    for r in (0, 99990, 399950, 2 ** 31 // k - 60, 539890):
        for e in range(experts):
            lo, hi = max(r, ends[e]), min(r + 100, ends[e + 1])
            if lo < hi:
                assert torch.equal(d[lo:hi], a[lo:hi].float() @ b[e * n:(e + 1) * n].float().T)
    say("gradient", m, n, k)
    da, db = H.MatmulGrad(m, n, k, experts=experts)(dd, a, b, offsets)
    for r in (0, 99950, 2 ** 31 // k - 60, 539890):
        for e in range(experts):
            lo, hi = max(r, ends[e]), min(r + 100, ends[e + 1])
            if lo < hi:
                assert torch.equal(da[lo:hi], (dd[lo:hi].float() @ b[e * n:(e + 1) * n].float()).to(torch.bfloat16))
    for e in range(experts):
        want = torch.zeros((n, k), device="cuda")
        for lo in range(ends[e], ends[e + 1], 65536):
            hi = min(lo + 65536, ends[e + 1])
            want += dd[lo:hi].float().T @ a[lo:hi].float()
        assert torch.equal(db[e * n:(e + 1) * n], want.to(torch.bfloat16)), e


def test_quantize_past_32_bits():
    """Rows whose every block holds 448 and whole numbers below 16: scales of 1,
    and e4m3 has them all."""
    rows, cols = 140000, 16384
    assert rows * cols > 2 ** 31
    x = whole((rows, cols), 7, 15)
    x[:, ::128] = 448
    say("quantize", rows, cols)
    y, scale = H.BlockQuantize(rows, cols)(x)
    assert (scale == 1).all()
    for r in (0, 2 ** 31 // cols - 50, rows - 100):
        assert torch.equal(y[r:r + 100].float(), x[r:r + 100].float())
    say("block product", rows, cols)
    b = whole((40, cols), 8, 1, torch.float8_e4m3fn)
    ones = torch.ones((1, cols // 128), device="cuda")
    d = H.Matmul(rows, 40, cols, "f8e4m3", scales="blocks", out_dtype="f32")(y, b, scale, ones)
    for r in (0, 2 ** 31 // cols - 50, rows - 100):
        assert torch.equal(d[r:r + 100], x[r:r + 100].float() @ b.float().T)
