"""The operators' refusals and plans (no GPU): every rule of the header's
operator section that create checks, through the binding and through raw
descriptors."""
import ctypes
import itertools

import numpy as np
import pytest
import torch

import compiler_hlo_amd as H
from compiler_hlo_amd import operators as O

MAKERS = {
    "rms_norm": lambda **k: H.RmsNorm(5, 64, mode="plan", **k),
    "rms_norm_grad": lambda **k: H.RmsNormGrad(5, 64, mode="plan", **k),
    "matmul": lambda **k: H.Matmul(5, 32, 64, mode="plan", **k),
    "matmul_grad": lambda **k: H.MatmulGrad(5, 32, 64, mode="plan", **k),
    "gated": lambda **k: H.GatedFeedForward(5, 32, 64, mode="plan", **k),
    "gated_grad": lambda **k: H.GatedFeedForwardGrad(5, 32, 64, mode="plan", **k),
    "dropout": lambda **k: H.Dropout(5, 64, mode="plan", **k),
}


def names(op):
    return [b.name for b in op.params], [b.name for b in op.results]


def dims(op):
    return {b.name: b.dims for b in op.params + op.results}


def test_buffers_in_order():
    op = H.RmsNorm(5, 64, residual=True, out_dtype="s8", mode="plan")
    assert names(op) == (["x", "weight", "residual"], ["y", "scale", "stream", "rstd"])
    op = H.RmsNormGrad(5, 64, stream_grad=True, mode="plan")
    assert names(op) == (["dy", "h", "weight", "rstd", "dstream"], ["dx", "dweight"])
    op = H.Matmul(5, 32, 64, "f8e4m3", bias=True, residual=True, save=True, activation="gelu", mode="plan")
    assert names(op) == (["a", "b", "a_scale", "b_scale", "bias", "residual"], ["d", "z"])
    assert dims(op)["b"] == (32, 64) and dims(op)["b_scale"] == (32,) and dims(op)["bias"] == (32,)
    op = H.MatmulGrad(5, 32, 64, bias=True, activation="relu", mode="plan")
    assert names(op) == (["dd", "a", "b", "z"], ["da", "db", "dbias"])
    op = H.GatedFeedForward(5, 32, 64, "s8", save=True, mode="plan")
    assert names(op) == (["a", "b", "a_scale", "b_scale"], ["d", "z"])
    assert dims(op)["b"] == (64, 64) and dims(op)["z"] == (5, 64) and dims(op)["b_scale"] == (64,)
    op = H.GatedFeedForwardGrad(5, 32, 64, mode="plan")
    assert names(op) == (["dd", "a", "b", "z"], ["da", "db"])
    op = H.Dropout(5, 64, residual=True, mode="plan")
    assert names(op) == (["x", "state", "residual"], ["y"])
    assert op.params[1].dtype == "s64" and dims(op)["state"] == (2,)


def test_algorithmic_counts():
    p = H.Matmul(7, 96, 160, "bf16", bias=True, residual=True, mode="plan").plan()
    assert p["algorithmic_bytes"] == 2 * (7 * 160 + 96 * 160 + 96 + 2 * 7 * 96)
    assert p["algorithmic_flops"] == 2 * 7 * 96 * 160
    p = H.GatedFeedForwardGrad(7, 96, 160, "f16", mode="plan").plan()
    assert p["algorithmic_bytes"] == 2 * (7 * 96 + 2 * 7 * 160 + 2 * 192 * 160 + 7 * 192)
    assert p["algorithmic_flops"] == 4 * 7 * 192 * 160


@pytest.mark.parametrize("make, status, text", [
    (lambda: H.RmsNorm(4, 0, mode="plan"), "HF_ERR_INVALID", "no elements"),
    (lambda: H.RmsNorm(-1, 8, mode="plan"), "HF_ERR_INVALID", "negative"),
    (lambda: H.RmsNorm(4, 8, eps=-1.0, mode="plan"), "HF_ERR_INVALID", "epsilon"),
    (lambda: H.RmsNorm(4, 8, eps=float("nan"), mode="plan"), "HF_ERR_INVALID", "epsilon"),
    (lambda: H.RmsNorm(4, 8, "s8", mode="plan"), "HF_ERR_UNSUPPORTED", "element type"),
    (lambda: H.RmsNorm(4, 8, "bf16", out_dtype="f16", mode="plan"), "HF_ERR_UNSUPPORTED", "results"),
    (lambda: H.RmsNorm(4, 8, "bf16", weight_dtype="f16", mode="plan"), "HF_ERR_INVALID", "weight"),
    (lambda: H.RmsNorm(2 ** 31, 8, mode="plan"), "HF_ERR_UNSUPPORTED", "2^31"),
    (lambda: H.RmsNormGrad(4, 8, "f8e4m3", mode="plan"), "HF_ERR_UNSUPPORTED", "element type"),
    (lambda: H.Matmul(4, 8, 8, "f32", mode="plan"), "HF_ERR_UNSUPPORTED", "operands"),
    (lambda: H.Matmul(4, 8, 8, "bf16", out_dtype="s8", mode="plan"), "HF_ERR_UNSUPPORTED", "results"),
    (lambda: H.Matmul(4, 8, 1 << 17, "s8", mode="plan"), "HF_ERR_UNSUPPORTED", "2^17"),
    (lambda: H.Matmul(4, 8, 1 << 22, "bf16", mode="plan"), "HF_ERR_UNSUPPORTED", "8 MB"),
    (lambda: H.Matmul(4, 8, -8, "bf16", mode="plan"), "HF_ERR_INVALID", "negative"),
    (lambda: H.MatmulGrad(4, 8, 8, "s8", mode="plan"), "HF_ERR_UNSUPPORTED", "operands"),
    (lambda: H.GatedFeedForward(4, 2 ** 30, 8, mode="plan"), "HF_ERR_UNSUPPORTED", "2n"),
    (lambda: H.GatedFeedForwardGrad(4, 8, 8, "f8e4m3", mode="plan"), "HF_ERR_UNSUPPORTED", "operands"),
    (lambda: H.Dropout(4, 8, p=1.0, mode="plan"), "HF_ERR_INVALID", "probability"),
    (lambda: H.Dropout(4, 8, p=-0.1, mode="plan"), "HF_ERR_INVALID", "probability"),
    (lambda: H.Dropout(4, 8, p=float("nan"), mode="plan"), "HF_ERR_INVALID", "probability"),
    (lambda: H.Dropout(4, 8, "s32", mode="plan"), "HF_ERR_UNSUPPORTED", "element type"),
    (lambda: H.Matmul(4, 8, 8, strides={"a": 7}, mode="plan"), "HF_ERR_INVALID", "row stride"),
    (lambda: H.Matmul(4, 8, 8, strides={"d": -8}, mode="plan"), "HF_ERR_INVALID", "row stride"),
    (lambda: H.Matmul(4, 8, 8, bias=True, strides={"bias": 16}, mode="plan"), "HF_ERR_INVALID", "vector"),
])
def test_refusals(make, status, text):
    with pytest.raises(H.FusionError) as e:
        make()
    assert e.value.status == status and text in e.value.message, e.value.message


def test_binding_refusals():
    with pytest.raises(ValueError, match="activation"):
        H.Matmul(4, 8, 8, activation="swish", mode="plan")
    with pytest.raises(ValueError, match="element type"):
        H.Matmul(4, 8, 8, "fp8", mode="plan")
    with pytest.raises(ValueError, match="no buffer"):
        H.Matmul(4, 8, 8, strides={"bias": 8}, mode="plan")


def raw(op, change):
    d = O.HfOperatorDesc(H.ABI_VERSION, O.KINDS[op], 4, 8, 8 if op not in ("rms_norm", "rms_norm_grad", "dropout")
                         else 0, 1, 1, 1, 0, 0, 1e-5, 0.1)
    change(d)
    h = ctypes.c_void_p()
    rc = H.library().hf_operator_create(ctypes.byref(d), H.PLAN_ONLY, ctypes.byref(h))
    text = H.library().hf_last_error().decode()
    if rc == 0:
        H.library().hf_operator_destroy(h)
    else:
        assert not h.value and text
    return H.STATUS[rc], text


@pytest.mark.parametrize("op", sorted(O.KINDS))
def test_raw_descriptor_refusals(op):
    def put(**kw):
        return lambda d: [setattr(d, k, v) for k, v in kw.items()]
    assert raw(op, put()) == ("HF_OK", "")
    for kw in (dict(abi_version=3), dict(kind=7), dict(kind=-1), dict(flags=8), dict(dtype=10), dict(dtype=-1),
               dict(out_dtype=99), dict(activation=4), dict(activation=-1)):
        assert raw(op, put(**kw))[0] == "HF_ERR_INVALID", kw

    def last(d):
        d.row_stride[O.MAX_BUFFERS - 1] = 64
    assert raw(op, last)[0] == "HF_ERR_INVALID"
    if op in ("rms_norm", "rms_norm_grad", "dropout"):
        assert raw(op, put(k=1))[0] == "HF_ERR_INVALID"
        assert raw(op, put(activation=1))[0] == "HF_ERR_INVALID"
        assert raw(op, put(flags=O.BIAS))[0] == "HF_ERR_INVALID"


def test_null_arguments():
    lib = H.library()
    d = O.HfOperatorDesc(H.ABI_VERSION, 0, 4, 8, 0, 1, 1, 1, 0, 0, 1e-5, 0.0)
    h = ctypes.c_void_p()
    assert lib.hf_operator_create(ctypes.byref(d), 0, None) == 1
    assert lib.hf_operator_create(None, 0, ctypes.byref(h)) == 1
    assert lib.hf_operator_create(ctypes.byref(d), 64, ctypes.byref(h)) == 1
    assert lib.hf_operator_plan(None, None) == 1
    assert lib.hf_operator_launch(None, None, 0, None, 0, None, None) == 1
    assert lib.hf_operator_launch_noalloc(None, None, 0, None, 0, None) == 1
    assert lib.hf_operator_destroy(None) == 0


@pytest.mark.parametrize("name", sorted(MAKERS))
def test_a_plan_only_handle_refuses_to_launch(name):
    op = MAKERS[name]()
    with pytest.raises(H.FusionError) as e:
        op.launch_ptrs([0] * len(op.params), [0] * len(op.results))
    assert e.value.status == "HF_ERR_INVALID" and "plan-only" in e.value.message
    op.close()
    op.close()


def test_mutated_descriptors_never_crash():
    """Random, mostly out-of-range fields: create answers with a status."""
    g = np.random.Generator(np.random.PCG64(11))
    wild = [-2 ** 63, -1, 0, 1, 2, 3, 7, 8, 63, 64, 100, 2 ** 17, 2 ** 31 - 1, 2 ** 31, 2 ** 40, 2 ** 63 - 1]
    seen = set()
    for _ in range(4000):
        d = O.HfOperatorDesc(H.ABI_VERSION, int(g.integers(0, 7)), 4, 8, 8, 1, 1, 1, 0, 0, 1e-5, 0.1)
        if d.kind in (0, 1, 6):
            d.k = 0
        for _ in range(int(g.integers(1, 4))):
            f = g.choice(["kind", "m", "n", "k", "dtype", "out_dtype", "weight_dtype", "activation", "flags",
                          "epsilon", "probability", "row_stride"])
            v = wild[int(g.integers(0, len(wild)))]
            if f == "row_stride":
                d.row_stride[int(g.integers(0, O.MAX_BUFFERS))] = v
            elif f in ("m", "n", "k"):
                setattr(d, f, v)
            elif f in ("epsilon", "probability"):
                setattr(d, f, float(g.choice([0.0, 0.5, 1.0, -1.0, np.inf, np.nan, 1e300])))
            else:
                setattr(d, f, int(np.array(v % 2 ** 32, np.uint32).view(np.int32)) if f != "flags" else v % 2 ** 32)
        h = ctypes.c_void_p()
        rc = H.library().hf_operator_create(ctypes.byref(d), H.PLAN_ONLY, ctypes.byref(h))
        assert rc in (0, 1, 2)
        seen.add(rc)
        if rc == 0:
            info = O.HfOperatorInfo()
            assert H.library().hf_operator_plan(h, ctypes.byref(info)) == 0
            assert info.workspace_bytes >= 0
            H.library().hf_operator_destroy(h)
    assert seen == {0, 1, 2}


def test_generator_against_published_vectors():
    """The counter-based generator's definition, in numpy as the GPU tests use
    it, against the known answers published with Philox4x32-10 (counter and
    key all zero, all one)."""
    from operators_reference import philox
    assert [hex(int(w)) for w in philox(np.zeros(1, np.uint64), 0)[0]] == \
        ["0x6627e8d5", "0xe169c58d", "0xbc57ac4c", "0x9b00dbd8"]


def test_workspace_is_bounded_by_the_operands():
    """The gradients keep dz and copies of operands whose rows do not start on
    16 bytes; nothing grows with the product of three sizes."""
    for m, n, k, half in itertools.product((1, 129, 4096), (8, 1001, 4096), (8, 999, 4096), ("bf16", "f16")):
        ws = H.MatmulGrad(m, n, k, half, activation="gelu", bias=True, mode="plan").workspace_bytes
        pad = lambda v: -(-v // 8) * 8
        packed = 2 * (pad(n) * m + pad(k) * (m + n)) + 4 * 512 * n
        partial = 16 * 4 * (m * pad(k) + n * pad(k))
        assert ws <= packed + partial + 4096


@pytest.mark.parametrize("m, n, k, dtype, want", [
    (1, 4096, 16384, "bf16", (16, 16, 1)),     # few rows: registers, 256 column groups of 16 waves
    (8, 512, 16384, "bf16", (16, 16, 4)),      # too few column groups: the contraction over workgroups too
    (9, 4096, 4096, "bf16", (64, 128, 4)),     # strips, shared by 4 workgroups
    (64, 22528, 4096, "bf16", (64, 128, 1)),
    (1, 22528, 4096, "bf16", (64, 128, 1)),    # enough columns for strips from one row on
    (65, 64, 64, "bf16", (128, 128, 1)),       # tiles
    (1024, 4096, 4096, "bf16", (128, 128, 1)),
    (256, 4096, 4096, "bf16", (128, 128, 4)),  # shared by 4 workgroups
    (8192, 8192, 8192, "bf16", (256, 256, 1)),
    (4096, 4096, 16384, "f8e4m3", (256, 256, 1)),
])
def test_tile_and_split_choices(m, n, k, dtype, want):
    """The kernels chosen for shapes that were measured."""
    p = H.Matmul(m, n, k, dtype, mode="plan").plan()
    assert (p["tile_rows"], p["tile_cols"], p["splits"]) == want
    assert (p["workspace_bytes"] > 0) == (want[2] > 1)


@pytest.mark.parametrize("make", [
    lambda: H.Matmul(2 ** 30, 129, 8, "f8e4m3", out_dtype="bf16", mode="plan"),
    lambda: H.GatedFeedForward(2 ** 30, 65, 8, "f8e4m3", out_dtype="bf16", mode="plan"),
    lambda: H.MatmulGrad(2 ** 30, 1, 600, mode="plan"),
    lambda: H.Matmul(2 ** 26, 2 ** 26, 2 ** 21, mode="plan"),
])
def test_more_tiles_than_a_launch_holds(make):
    """Refused at create, not by the runtime at launch."""
    with pytest.raises(H.FusionError) as e:
        make()
    assert e.value.status == "HF_ERR_UNSUPPORTED" and "tiles" in e.value.message, e.value.message


def test_the_largest_sizes_plan():
    for op in (H.RmsNorm(2 ** 31 - 256, 64, mode="plan"), H.Dropout(2 ** 31 - 256, 4096, mode="plan"),
               H.RmsNormGrad(1, 2 ** 30, mode="plan"), H.Matmul(1, 2 ** 30, 8, mode="plan"),
               H.Matmul(2 ** 30, 64, 64, mode="plan"), H.MatmulGrad(2 ** 30, 64, 64, mode="plan")):
        assert op.plan()["algorithmic_flops"] >= 0


def test_a_bound_launch_after_close_is_refused():
    """The binding's object keeps no handle that has been destroyed."""
    op = H.Matmul(4, 8, 16, mode="plan")

    class Stream:
        cuda_stream = 0
    tensors = [torch.zeros(b.dims, dtype=torch.bfloat16) for b in op.params + op.results]
    launch = O.BoundLaunch(op, tensors[:2], tensors[2:], None)
    with pytest.raises(H.FusionError) as e:
        launch(Stream)
    assert "plan-only" in e.value.message
    op.close()
    for call in (lambda: launch(Stream), lambda: op.launch_ptrs([0, 0], [0])):
        with pytest.raises(H.FusionError) as e:
            call()
        assert e.value.status == "HF_ERR_INVALID" and "NULL handle" in e.value.message
    op.close()
