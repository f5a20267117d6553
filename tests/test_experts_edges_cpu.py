"""Plans of the operators by expert at many experts and short features (no GPU)."""
import pytest

import compiler_hlo_amd as H


@pytest.mark.parametrize("m, n, k, experts, want", [
    (8192, 128, 128, 127, 128),
    (8192, 128, 128, 128, 128),     # a large tile would be a quarter full
    (8192, 128, 128, 256, 128),
    (8192, 48, 64, 200, 128),
    (8192, 384, 384, 64, 128),      # 4 large tiles an expert for 9 small ones
    (16384, 640, 384, 60, 128),
    (8192, 136, 136, 200, 256),     # as many sums in either
    (8192, 256, 256, 128, 256),
    (16384, 4096, 1408, 16, 256),   # 6 large tiles' columns for 11 small ones'
    (16384, 4096, 1152, 16, 256),
    (16384, 4096, 1100, 16, 256),
    (16384, 4096, 1000, 16, 256),
    (16384, 4096, 640, 16, 128),
])
def test_a_gradients_tiles_are_not_mostly_padding(m, n, k, experts, want):
    assert H.MatmulGrad(m, n, k, experts=experts, mode="plan").plan()["tile_rows"] == want
    if n % 2 == 0:  # gated: 2n rows of db an expert
        assert H.GatedFeedForwardGrad(m, n // 2, k, experts=experts, mode="plan").plan()["tile_rows"] == want
