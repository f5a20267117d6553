"""The operators by expert and with block scales at the ends of their ranges:
rows of no columns, scales at the ends of f32, many experts."""
import pytest
import torch

import compiler_hlo_amd as H
import experts_reference as X
import operators_reference as R
from test_operators_gpu import T, gen, say

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["s8", "f8e4m3"])
def test_dispatch_of_no_columns_sends_the_scales(dtype):
    """A row's scale is its own result: it is sent though the row is empty."""
    for tokens, top_k in ((4, 2), (300, 3)):
        say("dispatch of no columns", dtype, tokens, top_k)
        g = gen(tokens)
        place, order, _ = X.sort(torch.randint(-1, 5, (tokens, top_k), generator=g, dtype=torch.int32), 5)
        n = int((order >= 0).sum())
        scale = torch.rand(tokens, generator=g)
        y, s = H.ExpertDispatch(tokens, top_k, 0, dtype)(
            torch.empty((tokens, 0), dtype=T[dtype], device="cuda"), place.cuda(), scale.cuda(),
            out=[torch.empty((tokens * top_k, 0), dtype=T[dtype], device="cuda"), torch.full((tokens * top_k,), -7.0, device="cuda")])
        assert y.shape == (tokens * top_k, 0)
        assert torch.equal(s[:n].cpu(), scale[order[:n].long() // top_k]) and (s[n:] == -7.0).all()


def test_dispatch_of_no_columns_in_blocks_writes_nothing():
    y, s = H.ExpertDispatch(4, 2, 0, "f8e4m3", scales="blocks")(
        torch.empty((4, 0), dtype=T["f8e4m3"], device="cuda"), torch.zeros((4, 2), dtype=torch.int32, device="cuda"),
        torch.empty((0, 4), device="cuda"))
    assert y.shape == (8, 0) and s.shape == (0, 8)
