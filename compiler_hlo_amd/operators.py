"""The operators of a transformer's feed-forward layer (hf_operator_* in
include/hlofusion.h): RmsNorm, Matmul, GatedFeedForward and Dropout, and the
gradients RmsNormGrad, MatmulGrad and GatedFeedForwardGrad.

Like a Fusion, an operator is an immutable handle for fixed sizes and types,
and this module marshals arguments only.  Creating one compiles nothing and
costs a few microseconds, so a program may make one for every batch size it
meets::

    import torch, compiler_hlo_amd as H

    norm = H.RmsNorm(rows, 4096, "bf16", residual=True, out_dtype="f8e4m3")
    q, scale, stream, rstd = norm(x, weight, residual)

    up = H.GatedFeedForward(rows, 11264, 4096, "f8e4m3", out_dtype="bf16")
    h = up(q, w, scale, w_scale)

Tensors are [rows, columns] with adjacent elements in a row.  ``strides=``
names buffers whose rows are further apart than their length, in elements:
``Matmul(m, n, k, "bf16", strides={"a": 8192})``.

``op(*params)`` launches on torch's current stream and returns the result
tensors; ``op.bind(*params)`` fixes the buffers, and calling the bound launch
again costs no marshalling.  An operator's gradient is an operator of its own:
nothing is recorded in torch's autograd graph.
"""
from __future__ import annotations

import ctypes

from . import (ABI_VERSION, COMPILE_ONLY, DTYPES, PLAN_ONLY, _check, _lib)

MAX_BUFFERS = 10
OPERATOR_DTYPES = dict(DTYPES, f8e4m3=8, s64=9)
_DTYPE_NAMES = {v: k for k, v in OPERATOR_DTYPES.items()}
KINDS = {"rms_norm": 0, "rms_norm_grad": 1, "matmul": 2, "matmul_grad": 3, "gated": 4, "gated_grad": 5,
         "dropout": 6}
ACTIVATIONS = {None: 0, "none": 0, "relu": 1, "gelu": 2, "silu": 3}
RESIDUAL, BIAS, SAVE = 1, 2, 4


class HfOperatorDesc(ctypes.Structure):
    _fields_ = [("abi_version", ctypes.c_int32), ("kind", ctypes.c_int32), ("m", ctypes.c_int64),
                ("n", ctypes.c_int64), ("k", ctypes.c_int64), ("dtype", ctypes.c_int32),
                ("out_dtype", ctypes.c_int32), ("weight_dtype", ctypes.c_int32),
                ("activation", ctypes.c_int32), ("flags", ctypes.c_uint32), ("epsilon", ctypes.c_double),
                ("probability", ctypes.c_double), ("row_stride", ctypes.c_int64 * MAX_BUFFERS)]


class HfBufferInfo(ctypes.Structure):
    _fields_ = [("dtype", ctypes.c_int32), ("rank", ctypes.c_int32), ("dims", ctypes.c_int64 * 2),
                ("row_stride", ctypes.c_int64)]


class HfOperatorInfo(ctypes.Structure):
    _fields_ = [("n_params", ctypes.c_int32), ("n_results", ctypes.c_int32),
                ("buffers", HfBufferInfo * MAX_BUFFERS), ("workspace_bytes", ctypes.c_int64),
                ("algorithmic_bytes", ctypes.c_int64), ("algorithmic_flops", ctypes.c_int64),
                ("tile_rows", ctypes.c_int32), ("tile_cols", ctypes.c_int32), ("splits", ctypes.c_int32)]


_lib.hf_operator_create.restype = ctypes.c_int
_lib.hf_operator_create.argtypes = [ctypes.POINTER(HfOperatorDesc), ctypes.c_uint32, ctypes.POINTER(ctypes.c_void_p)]
_lib.hf_operator_plan.restype = ctypes.c_int
_lib.hf_operator_plan.argtypes = [ctypes.c_void_p, ctypes.POINTER(HfOperatorInfo)]
_lib.hf_operator_launch.restype = ctypes.c_int
_lib.hf_operator_launch.argtypes = [ctypes.c_void_p, ctypes.POINTER(ctypes.c_void_p), ctypes.c_int32,
                                    ctypes.POINTER(ctypes.c_void_p), ctypes.c_int32, ctypes.c_void_p,
                                    ctypes.c_void_p]
# the same function with its array arguments as addresses: a bound launch
# passes integers, which ctypes converts faster than arrays (0.3 us a call)
_launch_addresses = _lib["hf_operator_launch"]
_launch_addresses.restype = ctypes.c_int
_launch_addresses.argtypes = [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int32, ctypes.c_void_p, ctypes.c_int32,
                              ctypes.c_void_p, ctypes.c_void_p]
_lib.hf_operator_launch_noalloc.restype = ctypes.c_int
_lib.hf_operator_launch_noalloc.argtypes = [ctypes.c_void_p, ctypes.POINTER(ctypes.c_void_p), ctypes.c_int32,
                                            ctypes.POINTER(ctypes.c_void_p), ctypes.c_int32, ctypes.c_void_p]
_lib.hf_operator_destroy.restype = ctypes.c_int
_lib.hf_operator_destroy.argtypes = [ctypes.c_void_p]


def _torch_dtype(name):
    import torch
    return {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16, "s8": torch.int8,
            "u8": torch.uint8, "s32": torch.int32, "f8e4m3": torch.float8_e4m3fn, "s64": torch.int64}[name]


class Buffer:
    """One parameter or result: its name, element type, dims and row stride."""

    def __init__(self, name, info):
        self.name = name
        self.dtype = _DTYPE_NAMES[info.dtype]
        self.dims = tuple(info.dims[:info.rank])
        self.row_stride = info.row_stride if info.rank == 2 else None
        self.numel = self.dims[0] * (self.dims[1] if info.rank == 2 else 1)
        self.extent = self.numel
        if info.rank == 2 and self.numel:
            self.extent = (self.dims[0] - 1) * self.row_stride + self.dims[1]

    def check(self, t):
        want = _torch_dtype(self.dtype)
        ok = t.is_cuda and t.dtype == want and tuple(t.shape) == self.dims
        if ok and self.numel:
            if len(self.dims) == 1:
                ok = self.dims[0] <= 1 or t.stride(0) == 1
            else:
                ok = (self.dims[1] <= 1 or t.stride(1) == 1) and (self.dims[0] <= 1 or t.stride(0) == self.row_stride)
        if not ok:
            raise ValueError("%s must be a GPU tensor of %s%s%s" % (
                self.name, want, list(self.dims),
                "" if self.row_stride is None else ", rows %d elements apart" % self.row_stride))

    def empty(self, device):
        import torch
        t = torch.empty(self.extent, dtype=_torch_dtype(self.dtype), device=device)
        if len(self.dims) == 1:
            return t
        return t.as_strided(self.dims, (self.row_stride, 1))


class BoundLaunch:
    """hf_operator_launch with its buffers fixed (see Operator.bind); it keeps
    the operator and the tensors alive.  Calling it launches once more, on
    `stream` (a torch stream; None: the current one), and returns the same
    result tensors.  The buffers belong to the stream they were made on: a
    program that launches on another orders the two itself, and keeps this
    object until the launch has run."""

    def __init__(self, op, params, results, workspace):
        import torch
        self._op, self._params, self._workspace = op, params, workspace
        self.results = results[0] if len(results) == 1 else tuple(results)
        self._p = (ctypes.c_void_p * max(1, len(params)))(*[t.data_ptr() for t in params])
        self._r = (ctypes.c_void_p * len(results))(*[t.data_ptr() for t in results])
        # the handle as the operator's own object, which close() empties
        self._args = (op._h, ctypes.addressof(self._p), len(params), ctypes.addressof(self._r), len(results),
                      None if workspace is None else workspace.data_ptr())
        self._index = params[0].device.index
        self._launch = _launch_addresses
        self._current = torch._C._cuda_getCurrentRawStream

    def __call__(self, stream=None):
        rc = self._launch(*self._args, self._current(self._index) if stream is None else stream.cuda_stream)
        if rc:
            _check(rc)
        return self.results


class Operator:
    """Base of the operators; see the subclasses for what they compute and for
    their parameters and results in order.  ``mode`` is "load" (default) or
    "plan" (validate and plan only; no GPU)."""

    def __init__(self, kind, params, results, m, n, k, dtype, out_dtype, *, weight_dtype=None, activation=None,
                 flags=0, epsilon=0.0, probability=0.0, strides=None, mode="load"):
        if activation not in ACTIVATIONS:
            raise ValueError("activation must be one of %s" % sorted(a for a in ACTIVATIONS if a))
        for t in (dtype, out_dtype, weight_dtype or dtype):
            if t not in OPERATOR_DTYPES:
                raise ValueError("unknown element type %r" % (t,))
        names = params + results
        d = HfOperatorDesc(ABI_VERSION, KINDS[kind], m, n, k, OPERATOR_DTYPES[dtype], OPERATOR_DTYPES[out_dtype],
                           OPERATOR_DTYPES[weight_dtype or dtype], ACTIVATIONS[activation], flags, epsilon,
                           probability)
        for name, v in (strides or {}).items():
            if name not in names:
                raise ValueError("no buffer %r; this operator has %s" % (name, ", ".join(names)))
            d.row_stride[names.index(name)] = v
        h = ctypes.c_void_p()
        _check(_lib.hf_operator_create(ctypes.byref(d), {"load": 0, "compile": COMPILE_ONLY, "plan": PLAN_ONLY}[mode],
                                       ctypes.byref(h)))
        self._h = h
        info = HfOperatorInfo()
        _check(_lib.hf_operator_plan(h, ctypes.byref(info)))
        self._info = info
        buffers = [Buffer(name, info.buffers[i]) for i, name in enumerate(names)]
        self.params, self.results = buffers[:info.n_params], buffers[info.n_params:]
        self.workspace_bytes = info.workspace_bytes

    def plan(self) -> dict:
        """What the planner chose."""
        i = self._info
        return {f: getattr(i, f) for f in ("workspace_bytes", "algorithmic_bytes", "algorithmic_flops", "tile_rows",
                                           "tile_cols", "splits")}

    def _buffers(self, params, out, stream, workspace):
        import torch
        if len(params) != len(self.params):
            raise ValueError("expected %d parameters (%s), got %d" % (
                len(self.params), ", ".join(b.name for b in self.params), len(params)))
        for b, t in zip(self.params, params):
            b.check(t)
        if out is not None:
            out = [out] if isinstance(out, torch.Tensor) else list(out)
            if len(out) != len(self.results):
                raise ValueError("expected %d results (%s), got %d" % (
                    len(self.results), ", ".join(b.name for b in self.results), len(out)))
            for b, t in zip(self.results, out):
                b.check(t)
        device = params[0].device
        with torch.cuda.stream(stream):
            if out is None:
                out = [b.empty(device) for b in self.results]
            if workspace is None and self.workspace_bytes:
                workspace = torch.empty(self.workspace_bytes, dtype=torch.uint8, device=device)
        if workspace is not None and (not workspace.is_cuda or not workspace.is_contiguous()
                                      or workspace.numel() * workspace.element_size() < self.workspace_bytes):
            raise ValueError("workspace must be a dense GPU tensor of at least %d bytes" % self.workspace_bytes)
        return out, workspace

    def bind(self, *params, out=None, stream=None, workspace=None) -> BoundLaunch:
        """A launch with fixed buffers; those not given are allocated here."""
        out, workspace = self._buffers(params, out, stream, workspace)
        return BoundLaunch(self, params, out, workspace)

    def __call__(self, *params, out=None, stream=None, workspace=None):
        """Run on torch tensors; returns the result tensor, or a tuple of them.
        Results and a workspace that are not given come from torch's allocator
        on the launch stream.  With a `stream`, the program orders it after
        whatever fills the parameters, and may drop the tensors at once: the
        allocator is told of their use."""
        out, workspace = self._buffers(params, out, stream, workspace)
        if stream is not None:
            for t in (*params, *out, *([] if workspace is None else [workspace])):
                t.record_stream(stream)
        return BoundLaunch(self, params, out, workspace)(stream)

    def launch_ptrs(self, param_ptrs, result_ptrs, stream: int = 0, workspace: int = 0):
        """Launch with raw device pointers (ints) on a raw hipStream_t."""
        p = (ctypes.c_void_p * max(1, len(param_ptrs)))(*param_ptrs)
        r = (ctypes.c_void_p * max(1, len(result_ptrs)))(*result_ptrs)
        _check(_lib.hf_operator_launch(self._h, p, len(param_ptrs), r, len(result_ptrs), workspace or None, stream))

    def launch_noalloc_ptrs(self, param_ptrs, result_ptrs, stream: int = 0):
        """hf_operator_launch_noalloc: the library's per-GPU scratch memory
        stands in for the workspace (launches that overlap on one GPU race on
        it)."""
        p = (ctypes.c_void_p * max(1, len(param_ptrs)))(*param_ptrs)
        r = (ctypes.c_void_p * max(1, len(result_ptrs)))(*result_ptrs)
        _check(_lib.hf_operator_launch_noalloc(self._h, p, len(param_ptrs), r, len(result_ptrs), stream))

    def close(self):
        """Destroy the handle; launches of it, bound ones too, are refused from
        then on."""
        if getattr(self, "_h", None):
            h = ctypes.c_void_p(self._h.value)
            self._h.value = None  # in the bound launches' arguments too
            _check(_lib.hf_operator_destroy(h))

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def _eight(dtype):
    return dtype in ("s8", "f8e4m3")


class RmsNorm(Operator):
    """h = x + residual; y = h / sqrt(mean(h^2) + eps) * weight over each row.

    params: x [rows, cols], weight [cols], residual [rows, cols] (residual=True)
    results: y, scale [rows] (out_dtype "s8" or "f8e4m3": y is in units of its
    row's scale), stream = h (residual=True), rstd [rows]

    With a weight of ones and an 8-bit result it quantises rows for an 8-bit
    product: h = y * (scale / rstd)."""

    def __init__(self, rows, cols, dtype="bf16", *, residual=False, out_dtype=None, weight_dtype=None, eps=1e-5,
                 strides=None, mode="load"):
        out_dtype = out_dtype or dtype
        super().__init__("rms_norm", ["x", "weight"] + ["residual"] * residual,
                         ["y"] + ["scale"] * _eight(out_dtype) + ["stream"] * residual + ["rstd"],
                         rows, cols, 0, dtype, out_dtype, weight_dtype=weight_dtype, epsilon=eps,
                         flags=RESIDUAL * residual, strides=strides, mode=mode)


class RmsNormGrad(Operator):
    """The gradient of RmsNorm's y (and, with stream_grad, of its stream).

    params: dy, h (x, or the stream), weight, rstd, dstream (stream_grad=True)
    results: dx (the gradient of x and of the residual alike), dweight [cols] f32"""

    def __init__(self, rows, cols, dtype="bf16", *, stream_grad=False, weight_dtype=None, strides=None, mode="load"):
        super().__init__("rms_norm_grad", ["dy", "h", "weight", "rstd"] + ["dstream"] * stream_grad,
                         ["dx", "dweight"], rows, cols, 0, dtype, dtype, weight_dtype=weight_dtype,
                         flags=RESIDUAL * stream_grad, strides=strides, mode=mode)


class Matmul(Operator):
    """d = activation(a @ b.T * a_scale[:, None] * b_scale + bias) + residual.

    params: a [m, k], b [n, k], a_scale [m], b_scale [n] (dtype "s8" or
    "f8e4m3"), bias [n] (bias=True), residual [m, n] (residual=True)
    results: d [m, n], z [m, n] (save=True: before the activation, for MatmulGrad)"""

    def __init__(self, m, n, k, dtype="bf16", *, out_dtype=None, bias=False, activation=None, residual=False,
                 save=False, strides=None, mode="load"):
        out_dtype = out_dtype or ("bf16" if _eight(dtype) else dtype)
        super().__init__("matmul", ["a", "b"] + ["a_scale", "b_scale"] * _eight(dtype) + ["bias"] * bias
                         + ["residual"] * residual, ["d"] + ["z"] * save, m, n, k, dtype, out_dtype,
                         activation=activation, flags=RESIDUAL * residual + BIAS * bias + SAVE * save,
                         strides=strides, mode=mode)


class MatmulGrad(Operator):
    """The gradient of Matmul.  The residual's gradient is dd itself.  The
    gradient before the activation is rounded to dtype on its way into the
    products: a program in f16 scales its loss so that it fits f16's range.

    params: dd [m, n], a [m, k], b [n, k], z [m, n] (with an activation)
    results: da, db, dbias [n] f32 (bias=True)"""

    def __init__(self, m, n, k, dtype="bf16", *, bias=False, activation=None, strides=None, mode="load"):
        super().__init__("matmul_grad", ["dd", "a", "b"] + ["z"] * (ACTIVATIONS.get(activation, 1) != 0),
                         ["da", "db"] + ["dbias"] * bias, m, n, k, dtype, dtype, activation=activation,
                         flags=BIAS * bias, strides=strides, mode=mode)


class GatedFeedForward(Operator):
    """d = activation(a @ gate.T) * (a @ up.T) in one kernel; b holds the n
    gate channels' rows, then the n up channels'.

    params: a [m, k], b [2n, k], a_scale [m], b_scale [2n] (dtype "s8" or "f8e4m3")
    results: d [m, n], z [m, 2n] (save=True: both products, for the gradient)"""

    def __init__(self, m, n, k, dtype="bf16", *, out_dtype=None, activation="silu", save=False, strides=None,
                 mode="load"):
        out_dtype = out_dtype or ("bf16" if _eight(dtype) else dtype)
        super().__init__("gated", ["a", "b"] + ["a_scale", "b_scale"] * _eight(dtype), ["d"] + ["z"] * save,
                         m, n, k, dtype, out_dtype, activation=activation, flags=SAVE * save, strides=strides,
                         mode=mode)


class GatedFeedForwardGrad(Operator):
    """The gradient of GatedFeedForward.  The gradients of gate and up are
    rounded to dtype on their way into the products, as MatmulGrad's is.

    params: dd [m, n], a [m, k], b [2n, k], z [m, 2n]
    results: da [m, k], db [2n, k]"""

    def __init__(self, m, n, k, dtype="bf16", *, activation="silu", strides=None, mode="load"):
        super().__init__("gated_grad", ["dd", "a", "b", "z"], ["da", "db"], m, n, k, dtype, dtype,
                         activation=activation, strides=strides, mode=mode)


class Dropout(Operator):
    """y = keep * x / (1 - p) + residual.  The mask comes from a counter and is
    stored nowhere: the backward pass is this operator, without residual, on
    the gradient with the same state.

    params: x [rows, cols], state (int64 [2] on the GPU: seed, offset),
    residual [rows, cols] (residual=True)
    results: y.  The call uses ceil(rows * cols / 8) counters from offset on."""

    def __init__(self, rows, cols, dtype="bf16", *, p=0.1, residual=False, strides=None, mode="load"):
        super().__init__("dropout", ["x", "state"] + ["residual"] * residual, ["y"], rows, cols, 0, dtype, dtype,
                         probability=p, flags=RESIDUAL * residual, strides=strides, mode=mode)
