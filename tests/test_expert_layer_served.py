"""examples/expert_layer.py: how near the served layer is to the trained one."""
import os
import sys

import pytest
import torch

import operators_reference as R
from test_expert_layer_example import made

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
import expert_layer as E  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("experts, hidden, inner", [(5, 256, 200), (3, 200, 130), (70, 128, 64)])
@pytest.mark.parametrize("tokens", [1, 5, 300])
def test_the_served_layer_is_within_its_roundings(tokens, experts, hidden, inner):
    """A value in e4m3 is off by an error uniform in half a step, 2^-4 of the power
    of two: 2^-4 / sqrt 3 of it in the mean square, 2^-5.3 of the value over evenly
    spread mantissas.  A row and a weight in each of gate and up, the product of
    both and the last weight are six such errors on the way of a term, all but
    independent: sqrt 6 * 2^-5.3 = 0.062 of the sum's norm.  2 sqrt 3 * 2^-5 = 0.108
    leaves room for the values below a block's normal range."""
    l = made(tokens, 2, experts, hidden, inner, "bf16")
    l.forward()
    y = E.Served(l.master, experts)(l.x, l.expert, l.share)
    added = R.f64(l.y) - R.f64(l.x)
    off = float((R.f64(y) - R.f64(l.y)).norm() / added.norm())
    assert off < 2 * 3 ** 0.5 * 2.0 ** -5, off
