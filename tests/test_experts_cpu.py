"""Refusals and plans of the operators by expert and with block scales (no
GPU), through the binding and through raw descriptors."""
import ctypes

import numpy as np
import pytest

import compiler_hlo_amd as H
from compiler_hlo_amd import operators as O

MAKERS = {
    "expert_sort": lambda **k: H.ExpertSort(5, 2, 8, mode="plan", **k),
    "expert_dispatch": lambda **k: H.ExpertDispatch(5, 2, 64, mode="plan", **k),
    "expert_combine": lambda **k: H.ExpertCombine(5, 2, 64, mode="plan", **k),
    "expert_combine_grad": lambda **k: H.ExpertCombineGrad(5, 2, 64, mode="plan", **k),
    "block_quantize": lambda **k: H.BlockQuantize(5, 64, mode="plan", **k),
    "matmul": lambda **k: H.Matmul(10, 32, 64, experts=8, mode="plan", **k),
    "matmul_grad": lambda **k: H.MatmulGrad(10, 32, 64, experts=8, mode="plan", **k),
    "gated": lambda **k: H.GatedFeedForward(10, 32, 64, experts=8, mode="plan", **k),
    "gated_grad": lambda **k: H.GatedFeedForwardGrad(10, 32, 64, experts=8, mode="plan", **k),
    "blocks": lambda **k: H.Matmul(10, 32, 64, "f8e4m3", scales="blocks", mode="plan", **k),
}


def names(op):
    return [b.name for b in op.params], [b.name for b in op.results]


def dims(op):
    return {b.name: b.dims for b in op.params + op.results}


def test_buffers_in_order():
    op = H.ExpertSort(5, 2, 8, mode="plan")
    assert names(op) == (["expert"], ["place", "order", "offsets"])
    assert dims(op) == {"expert": (5, 2), "place": (5, 2), "order": (10,), "offsets": (9,)}
    assert {b.dtype for b in op.params + op.results} == {"s32"}
    op = H.ExpertDispatch(5, 2, 300, "f8e4m3", scales="blocks", mode="plan")
    assert names(op) == (["x", "place", "x_scale"], ["y", "y_scale"])
    assert dims(op)["x_scale"] == (3, 5) and dims(op)["y_scale"] == (3, 10) and dims(op)["y"] == (10, 300)
    op = H.ExpertDispatch(5, 2, 300, "s8", mode="plan")
    assert dims(op)["x_scale"] == (5,) and dims(op)["y_scale"] == (10,)
    assert names(H.ExpertDispatch(5, 2, 300, mode="plan")) == (["x", "place"], ["y"])
    op = H.ExpertCombine(5, 2, 64, residual=True, mode="plan")
    assert names(op) == (["y", "place", "weight", "residual"], ["d"])
    assert names(H.ExpertCombine(5, 2, 64, weighted=False, mode="plan")) == (["y", "place"], ["d"])
    op = H.ExpertCombineGrad(5, 2, 64, mode="plan")
    assert names(op) == (["dd", "y", "place", "weight"], ["dy", "dweight"])
    op = H.BlockQuantize(5, 300, mode="plan")
    assert names(op) == (["x"], ["y", "scale"]) and dims(op)["scale"] == (3, 5)
    op = H.Matmul(10, 130, 300, "f8e4m3", scales="blocks", bias=True, residual=True, save=True, mode="plan")
    assert names(op) == (["a", "b", "a_scale", "b_scale", "bias", "residual"], ["d", "z"])
    assert dims(op)["a_scale"] == (3, 10) and dims(op)["b_scale"] == (2, 3)
    op = H.GatedFeedForward(10, 130, 300, "f8e4m3", scales="blocks", experts=4, save=True, mode="plan")
    assert names(op) == (["a", "b", "a_scale", "b_scale", "offsets"], ["d", "z"])
    assert dims(op)["b"] == (4 * 260, 300) and dims(op)["b_scale"] == (16, 3) and dims(op)["offsets"] == (5,)
    op = H.Matmul(10, 130, 300, "s8", experts=4, mode="plan")
    assert dims(op)["a_scale"] == (10,) and dims(op)["b_scale"] == (520,)
    op = H.MatmulGrad(10, 32, 64, activation="gelu", experts=4, mode="plan")
    assert names(op) == (["dd", "a", "b", "z", "offsets"], ["da", "db"])
    assert dims(op)["db"] == (128, 64)
    op = H.GatedFeedForwardGrad(10, 32, 64, experts=4, mode="plan")
    assert dims(op)["db"] == (256, 64) and dims(op)["da"] == (10, 64)


@pytest.mark.parametrize("make, status, text", [
    (lambda: H.ExpertSort(4, 0, 8, mode="plan"), "HF_ERR_INVALID", "top_k"),
    (lambda: H.ExpertSort(-4, 2, 8, mode="plan"), "HF_ERR_INVALID", "negative"),
    (lambda: H.ExpertSort(4, 2, 1025, mode="plan"), "HF_ERR_UNSUPPORTED", "1024"),
    (lambda: H.ExpertSort(2 ** 28, 8, 8, mode="plan"), "HF_ERR_UNSUPPORTED", "pairs"),
    (lambda: H.ExpertSort(4, 2 ** 40, 8, mode="plan"), "HF_ERR_UNSUPPORTED", "pairs"),
    (lambda: H.ExpertDispatch(4, 2, 8, "s32", mode="plan"), "HF_ERR_UNSUPPORTED", "element type"),
    (lambda: H.ExpertDispatch(4, 2, 8, "bf16", scales="blocks", mode="plan"), "HF_ERR_INVALID", "block scales"),
    (lambda: H.ExpertDispatch(4, 2, 8, "s8", scales="blocks", mode="plan"), "HF_ERR_INVALID", "block scales"),
    (lambda: H.ExpertDispatch(4, -2, 8, mode="plan"), "HF_ERR_INVALID", "top_k"),
    (lambda: H.ExpertCombine(4, 2, 8, "f8e4m3", mode="plan"), "HF_ERR_UNSUPPORTED", "element type"),
    (lambda: H.ExpertCombineGrad(4, 2, 8, "s8", mode="plan"), "HF_ERR_UNSUPPORTED", "element type"),
    (lambda: H.BlockQuantize(4, 8, "s8", mode="plan"), "HF_ERR_UNSUPPORTED", "element type"),
    (lambda: H.Matmul(4, 8, 8, "bf16", scales="blocks", mode="plan"), "HF_ERR_INVALID", "block scales"),
    (lambda: H.GatedFeedForward(4, 8, 8, "s8", scales="blocks", mode="plan"), "HF_ERR_INVALID", "block scales"),
    (lambda: H.Matmul(4, 8, 8, experts=2, bias=True, mode="plan"), "HF_ERR_UNSUPPORTED", "bias"),
    (lambda: H.Matmul(4, 8, 8, experts=2, residual=True, mode="plan"), "HF_ERR_UNSUPPORTED", "residual"),
    (lambda: H.MatmulGrad(4, 8, 8, experts=2, bias=True, mode="plan"), "HF_ERR_UNSUPPORTED", "bias"),
    (lambda: H.Matmul(4, 8, 8, experts=2000, mode="plan"), "HF_ERR_UNSUPPORTED", "1024"),
    (lambda: H.Matmul(4, 2 ** 28, 8, experts=64, mode="plan"), "HF_ERR_UNSUPPORTED", "weights"),
    (lambda: H.Matmul(2 ** 30, 2 ** 20, 8, experts=64, mode="plan"), "HF_ERR_UNSUPPORTED", "tiles"),
    (lambda: H.MatmulGrad(64, 2 ** 20, 2 ** 20, experts=1024, mode="plan"), "HF_ERR_UNSUPPORTED", "tiles"),
    (lambda: H.BlockQuantize(4, 8, strides={"y": 7}, mode="plan"), "HF_ERR_INVALID", "row stride"),
    (lambda: H.ExpertSort(4, 2, 8, strides={"order": 16}, mode="plan"), "HF_ERR_INVALID", "vector"),
])
def test_refusals(make, status, text):
    with pytest.raises(H.FusionError) as e:
        make()
    assert e.value.status == status and text in e.value.message, e.value.message


def test_binding_refusals():
    with pytest.raises(ValueError, match="experts"):
        H.Matmul(4, 8, 8, experts=0, mode="plan")
    with pytest.raises(ValueError, match="scales"):
        H.Matmul(4, 8, 8, "f8e4m3", scales="block", mode="plan")
    with pytest.raises(ValueError, match="scales"):
        H.ExpertDispatch(4, 2, 8, "f8e4m3", scales="tensor", mode="plan")


@pytest.mark.parametrize("name", sorted(MAKERS))
def test_a_plan_only_handle_refuses_to_launch(name):
    op = MAKERS[name]()
    with pytest.raises(H.FusionError) as e:
        op.launch_ptrs([0] * len(op.params), [0] * len(op.results))
    assert e.value.status == "HF_ERR_INVALID" and "plan-only" in e.value.message
    op.close()
    op.close()


def create(d):
    h = ctypes.c_void_p()
    rc = H.library().hf_operator_create_extended(ctypes.byref(d), H.PLAN_ONLY, ctypes.byref(h))
    if rc == 0:
        info = O.HfOperatorInfo()
        assert H.library().hf_operator_plan(h, ctypes.byref(info)) == 0 and info.workspace_bytes >= 0
        H.library().hf_operator_destroy(h)
    else:
        assert not h.value and H.library().hf_last_error()
    return H.STATUS[rc]


def raw(kind, /, **kw):
    d = O.HfOperatorExtendedDesc(O.HfOperatorDesc(H.ABI_VERSION, kind, 4, 8, 8 if 2 <= kind <= 5 else 0, 1, 1, 1, 0, 0,
                                                  1e-5, 0.1), 8 if 2 <= kind <= 5 or kind == 7 else 0,
                                 2 if 7 <= kind <= 10 else 0)
    if kind == 7:
        d.op.n = 0
    if kind == 11:
        d.op.out_dtype = 8
    for k, v in kw.items():
        setattr(d if k in ("experts", "top_k") else d.op, k, v)
    return create(d)


@pytest.mark.parametrize("kind", range(12))
def test_raw_descriptors(kind):
    assert raw(kind) == "HF_OK"
    for kw in (dict(abi_version=3), dict(kind=12), dict(kind=-1), dict(flags=32), dict(dtype=10), dict(out_dtype=-1),
               dict(experts=-1), dict(top_k=-1), dict(m=-1)):
        assert raw(kind, **kw) == "HF_ERR_INVALID", kw
    if not 2 <= kind <= 5 and kind != 7:
        assert raw(kind, experts=3) == "HF_ERR_INVALID"
    if not 7 <= kind <= 10:
        assert raw(kind, top_k=3) == "HF_ERR_INVALID"
    if kind == 7:
        assert raw(kind, experts=0) == "HF_ERR_INVALID" and raw(kind, n=1) == "HF_ERR_INVALID"
    if kind > 6:
        assert raw(kind, k=1) == "HF_ERR_INVALID" and raw(kind, activation=1) == "HF_ERR_INVALID"


@pytest.mark.parametrize("kind", range(7, 12))
def test_the_plain_create_takes_none_of_the_new_kinds(kind):
    d = O.HfOperatorDesc(H.ABI_VERSION, kind, 4, 8, 0, 1, 1, 1, 0, 0, 1e-5, 0.1)
    h = ctypes.c_void_p()
    assert H.library().hf_operator_create(ctypes.byref(d), H.PLAN_ONLY, ctypes.byref(h)) == 1 and not h.value


def test_an_extended_descriptor_plans_what_the_plain_one_does():
    d = O.HfOperatorDesc(H.ABI_VERSION, 2, 300, 640, 4096, 1, 1, 1, 2, O.RESIDUAL | O.BIAS, 0.0, 0.0)
    infos = []
    for make, desc in ((H.library().hf_operator_create, d),
                       (H.library().hf_operator_create_extended, O.HfOperatorExtendedDesc(d, 0, 0))):
        h, info = ctypes.c_void_p(), O.HfOperatorInfo()
        assert make(ctypes.byref(desc), H.PLAN_ONLY, ctypes.byref(h)) == 0
        assert H.library().hf_operator_plan(h, ctypes.byref(info)) == 0
        H.library().hf_operator_destroy(h)
        infos.append(bytes(info))
    assert infos[0] == infos[1]


def test_null_arguments():
    lib, h = H.library(), ctypes.c_void_p()
    d = O.HfOperatorExtendedDesc(O.HfOperatorDesc(H.ABI_VERSION, 7, 4, 0, 0, 1, 1, 1, 0, 0, 0.0, 0.0), 8, 2)
    assert lib.hf_operator_create_extended(ctypes.byref(d), H.PLAN_ONLY, None) == 1
    assert lib.hf_operator_create_extended(None, H.PLAN_ONLY, ctypes.byref(h)) == 1
    assert lib.hf_operator_create_extended(ctypes.byref(d), 64, ctypes.byref(h)) == 1


def test_mutated_descriptors_never_crash():
    """Random, mostly out-of-range fields: create answers with a status."""
    g = np.random.Generator(np.random.PCG64(12))
    wild = [-2 ** 63, -1, 0, 1, 2, 3, 7, 8, 63, 64, 100, 1024, 2 ** 17, 2 ** 31 - 1, 2 ** 31, 2 ** 40, 2 ** 63 - 1]
    seen = set()
    for _ in range(6000):
        kind = int(g.integers(0, 12))
        change = {}
        for _ in range(int(g.integers(1, 4))):
            f = str(g.choice(["m", "n", "k", "experts", "top_k", "dtype", "out_dtype", "flags", "activation"]))
            v = wild[int(g.integers(0, len(wild)))]
            if f in ("dtype", "out_dtype", "activation"):
                v = int(np.array(v % 2 ** 32, np.uint32).view(np.int32))
            elif f == "flags":
                v %= 2 ** 32
            change[f] = v
        seen.add(raw(kind, **change))
    assert seen == {"HF_OK", "HF_ERR_INVALID", "HF_ERR_UNSUPPORTED"}


def test_workspaces():
    """A sort of one chunk needs none; the others keep counts by chunk."""
    assert H.ExpertSort(1024, 8, 64, mode="plan").workspace_bytes == 0
    big = H.ExpertSort(2 ** 20, 8, 1024, mode="plan").workspace_bytes
    assert 0 < big <= 256 * 1024 * 4
    assert H.Matmul(4096, 512, 1024, experts=8, mode="plan").workspace_bytes == 0
    # rows of 1023 elements do not start on 16 bytes: copies of both operands
    assert H.Matmul(64, 16, 1023, experts=8, mode="plan").workspace_bytes >= 2 * 1024 * (64 + 128)


@pytest.mark.parametrize("m, n, experts, dtype, want", [
    (64, 2048, 64, "bf16", 64),        # a row an expert: strips
    (24 * 64, 2048, 64, "bf16", 64),
    (25 * 64, 2048, 64, "bf16", 128),
    (159 * 16, 4096, 16, "bf16", 128),
    (160 * 16, 4096, 16, "bf16", 256),
    (2048, 512, 8, "bf16", 128),       # too few large tiles
    (160 * 16, 4096, 16, "blocks", 128),
    (640 * 16, 4096, 16, "blocks", 256),
    (640 * 16, 4096, 16, "f32", 128),  # e4m3 through f16
    (7, 4096, 64, "bf16", 64),
])
def test_tile_choices_by_expert(m, n, experts, dtype, want):
    kw = {"bf16": {}, "blocks": dict(dtype="f8e4m3", scales="blocks"), "f32": dict(dtype="f8e4m3", out_dtype="f32")}[dtype]
    p = H.Matmul(m, n, 2048, experts=experts, mode="plan", **kw).plan()
    assert p["tile_rows"] == want and p["tile_cols"] == max(want, 128)


@pytest.mark.parametrize("m, n, k, experts, dtype, splits", [
    (1, 2048, 4096, 8, "bf16", 8),       # a token of 8 experts: 16 strips
    (128, 1408, 4096, 32, "bf16", 1),    # strips enough
    (200, 512, 4096, 4, "bf16", 16),
    (200, 512, 4096, 4, "blocks", 11),
    (200, 512, 4096, 4, "s8", 1),        # scales by the expert's rows: whole
    (16384, 4096, 4096, 8, "bf16", 1),
])
def test_shared_contractions_by_expert(m, n, k, experts, dtype, splits):
    kw = {"blocks": dict(dtype="f8e4m3", scales="blocks")}.get(dtype, dict(dtype=dtype))
    p = H.Matmul(m, n, k, experts=experts, mode="plan", **kw).plan()
    assert p["splits"] == splits and (p["workspace_bytes"] > 0) == (splits > 1)


def test_shared_contractions_of_gradients_by_expert():
    for m, n, k, experts, split in ((12, 3712, 320, 2, True), (5549, 128, 896, 1, True), (16384, 4096, 1408, 16, False),
                                    (100, 512, 512, 8, False)):
        assert (H.MatmulGrad(m, n, k, experts=experts, mode="plan").workspace_bytes > 0) == split


@pytest.mark.parametrize("n, k, experts, want", [(4096, 1408, 16, 256), (512, 512, 8, 128), (1024, 1024, 8, 256)])
def test_tile_choices_of_gradients_by_expert(n, k, experts, want):
    assert H.MatmulGrad(100, n, k, experts=experts, mode="plan").plan()["tile_rows"] == want
