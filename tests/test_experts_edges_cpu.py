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


@pytest.mark.parametrize("rows, dtype, want", [
    (159, "bf16", 128), (160, "bf16", 256),
    (191, "blocks", 128), (192, "blocks", 256), (512, "blocks", 256),
    (512, "f32", 128),   # block scales through f16 have no large tile
])
def test_the_rows_an_expert_from_which_tiles_are_large(rows, dtype, want):
    kw = {"bf16": {}, "blocks": dict(dtype="f8e4m3", scales="blocks"),
          "f32": dict(dtype="f8e4m3", scales="blocks", out_dtype="f32")}[dtype]
    for experts, n in ((16, 4096), (40, 2048)):
        assert H.Matmul(rows * experts, n, 2048, experts=experts, mode="plan", **kw).plan()["tile_rows"] == want
        assert H.GatedFeedForward(rows * experts, n // 2, 2048, experts=experts, mode="plan", **kw).plan()["tile_rows"] == want
