"""The feed-forward operators of a transformer layer, case by case: what each
one reads and writes, its plain form, and its value from the definition.

Four operators, each in its forward and its backward direction:

* ``norm``    root-mean-square norm of the residual stream (x + residual), with
              the result in the stream's type or in 8 bits with a scale a row;
* ``product`` d = act(a @ b.T * scales + bias) + residual;
* ``gated``   h = act(x @ gate.T) * (x @ up.T), both projections at once;
* ``dropout`` y = residual + keep * x / (1 - p), the mask drawn from a counter.

A case is a dict of plain values.  ``own`` chooses between the plain form and
the library's operators.
"""
import math

import numpy as np
import torch

own = False

TORCH = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16, "s8": torch.int8,
         "f8e4m3": torch.float8_e4m3fn}
BYTES = {"f32": 4, "bf16": 2, "f16": 2, "s8": 1, "f8e4m3": 1}
QMAX = {"s8": 127.0, "f8e4m3": 448.0}
EPS = 1e-5


# --------------------------------------------------------------------------
# cases
# --------------------------------------------------------------------------
def norm(name, rows, cols, dtype, out, residual):
    return {"name": name, "op": "norm", "rows": rows, "cols": cols, "dtype": dtype, "out": out, "residual": residual}


def norm_grad(name, rows, cols, dtype, residual):
    return {"name": name, "op": "norm_grad", "rows": rows, "cols": cols, "dtype": dtype, "residual": residual}


def product(name, m, n, k, dtype, out, bias, act, residual):
    return {"name": name, "op": "product", "m": m, "n": n, "k": k, "dtype": dtype, "out": out, "bias": bias,
            "act": act, "residual": residual}


def product_grad(name, m, n, k, dtype, bias, act):
    return {"name": name, "op": "product_grad", "m": m, "n": n, "k": k, "dtype": dtype, "bias": bias, "act": act}


def gated(name, m, n, k, dtype, out, act, save):
    return {"name": name, "op": "gated", "m": m, "n": n, "k": k, "dtype": dtype, "out": out, "act": act, "save": save}


def gated_grad(name, m, n, k, dtype, act):
    return {"name": name, "op": "gated_grad", "m": m, "n": n, "k": k, "dtype": dtype, "act": act}


def dropout(name, rows, cols, dtype, p, residual):
    return {"name": name, "op": "dropout", "rows": rows, "cols": cols, "dtype": dtype, "p": p, "residual": residual}


def listed():
    return [
        # one token's residual stream before an 8-bit layer: the shortest call of a decode step
        norm("norm_token_f8", 1, 4096, "bf16", "f8e4m3", True),
        # the prompt of one request, an odd number of tokens, quantised for 8-bit products
        norm("norm_prompt_f8", 4099, 4096, "bf16", "f8e4m3", True),
        # the norm's backward pass in a training step, with the gradient that comes down the stream
        norm_grad("norm_backward_bf16", 16384, 4096, "bf16", True),
        # the down projection of a single token, added to the residual stream: bound by the weights
        product("product_token_bf16", 1, 4096, 16384, "bf16", "bf16", False, "none", True),
        # the down projection of a prompt in 8 bits with row and channel scales, odd number of tokens
        product("product_prompt_f8", 4099, 4096, 16384, "f8e4m3", "bf16", False, "none", True),
        # an up projection with bias and GELU, the backward pass of a training step
        product_grad("product_backward_bf16", 8192, 16384, 4096, "bf16", True, "gelu"),
        # gate and up projections of a decode batch: bound by the two weights
        gated("gated_batch_bf16", 24, 11264, 4096, "bf16", "bf16", "silu", False),
        # gate and up projections of a training step or a long prompt, pre-activations kept
        gated("gated_prompt_bf16", 8191, 11264, 4096, "bf16", "bf16", "silu", True),
        # their backward pass
        gated_grad("gated_backward_bf16", 4096, 11264, 4096, "bf16", "silu"),
        # a small activation in half precision: launch latency
        dropout("dropout_small_f16", 65, 1024, "f16", 0.1, False),
        # the output of a block added to the stream in a training step
        dropout("dropout_residual_bf16", 16384, 4096, "bf16", 0.1, True),
        # the same mask over a gradient in f32 with rows of an odd length
        dropout("dropout_backward_f32", 8191, 4097, "f32", 0.25, False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _dims(rng, lo, hi, step):
    return step * max(1, _log(rng, lo, hi) // step)


def draw(rng):
    op = rng.choice(["norm", "norm_grad", "product", "product_grad", "gated", "gated_grad", "dropout"])
    half = rng.choice(["bf16", "bf16", "f16"])
    if op in ("norm", "norm_grad", "dropout"):
        rows, cols = _log(rng, 1, 16384), _log(rng, 64, 16384)
        if rng.random() < 0.7:
            cols = 16 * max(4, cols // 16)
        rows = max(1, min(rows, 16384 * 4096 // cols))
        dtype = rng.choice([half, half, half, "f32"])
        residual = rng.random() < 0.6
        if op == "norm":
            return norm("", rows, cols, dtype, rng.choice([dtype, "f8e4m3"]), residual) | {"name": "drawn"}
        if op == "norm_grad":
            return norm_grad("", rows, cols, dtype, residual) | {"name": "drawn"}
        return dropout("", rows, cols, dtype, rng.choice([0.05, 0.1, 0.25, 0.5]), residual) | {"name": "drawn"}
    # token counts of every size; features mostly in steps of 64, sometimes odd
    step = rng.choice([64, 64, 64, 8, 1])
    m, n, k = _log(rng, 1, 8192), _dims(rng, 256, 11264, step), _dims(rng, 256, 16384, step)
    act = rng.choice(["silu", "gelu"])
    if op == "gated":
        k = min(k, 4096)
        dtype = rng.choice([half, "f8e4m3", "s8"])
        return gated("", m, n, k, dtype, half, act, rng.random() < 0.5) | {"name": "drawn"}
    if op == "gated_grad":
        m, k = min(m, 4096), min(k, 4096)
        return gated_grad("", m, n, k, half, act) | {"name": "drawn"}
    act = rng.choice(["none", "relu", "gelu", "silu"])
    if op == "product":
        dtype = rng.choice([half, "f8e4m3", "s8"])
        return product("", m, n, k, dtype, half, rng.random() < 0.5, act, rng.random() < 0.5) | {"name": "drawn"}
    m = min(m, 4096)
    return product_grad("", m, n, min(k, 4096), half, rng.random() < 0.5, act) | {"name": "drawn"}


# --------------------------------------------------------------------------
# inputs
# --------------------------------------------------------------------------
def _normal(gen, shape, sigma, dtype):
    return (torch.randn(shape, generator=gen, device="cuda") * sigma).to(TORCH[dtype])


def _weight(gen, rows, k, dtype):
    """A weight of `rows` output channels: N(0, 1/k), in 8 bits with a scale a channel."""
    return _eight(torch.randn((rows, k), generator=gen, device="cuda") / math.sqrt(k), dtype)


def _eight(x, dtype):
    """x in `dtype`; in 8 bits with a scale a row (the largest magnitude of a row on the largest value)."""
    if dtype not in QMAX:
        return x.to(TORCH[dtype]), None
    scale = x.abs().amax(1) / QMAX[dtype]
    q = x / scale[:, None]
    return (q.round() if dtype == "s8" else q).clamp(-QMAX[dtype], QMAX[dtype]).to(TORCH[dtype]), scale


def _inputs(case, seed):
    """The inputs of a case by name, in the order in which the operator takes them."""
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    op, t = case["op"], case["dtype"]
    if op == "norm":
        shape = (case["rows"], case["cols"])
        d = {"x": _normal(g, shape, 1.0, t), "weight": _normal(g, shape[1:], 0.1, "f32").add_(1).to(TORCH[t])}
        if case["residual"]:
            d["residual"] = _normal(g, shape, 2.0, t)
        return d
    if op == "norm_grad":
        shape = (case["rows"], case["cols"])
        h = _normal(g, shape, 2.0, t)
        d = {"dy": _normal(g, shape, 0.02, t), "h": h,
             "weight": _normal(g, shape[1:], 0.1, "f32").add_(1).to(TORCH[t]),
             "rstd": (h.double().square().mean(1) + EPS).rsqrt().float()}
        if case["residual"]:
            d["dstream"] = _normal(g, shape, 0.02, t)
        return d
    if op == "dropout":
        shape = (case["rows"], case["cols"])
        d = {"x": _normal(g, shape, 1.0, t),
             "state": torch.tensor([int(seed) * 7919 + 1234567890123, int(seed) * 4096 + (1 << 32) - 77], device="cuda")}
        if case["residual"]:
            d["residual"] = _normal(g, shape, 2.0, t)
        return d
    m, n, k = case["m"], case["n"], case["k"]
    wide = n if op.startswith("product") else 2 * n
    if op in ("product", "gated"):
        a, sa = _eight(torch.randn((m, k), generator=g, device="cuda"), t)
        b, sb = _weight(g, wide, k, t)
        d = {"a": a, "b": b}
        if sa is not None:
            d |= {"a_scale": sa, "b_scale": sb}
        if case.get("bias"):
            d["bias"] = _normal(g, (n,), 0.1, case["out"])
        if case.get("residual"):
            d["residual"] = _normal(g, (m, n), 2.0, case["out"])
        return d
    d = {"dd": _normal(g, (m, n), 0.02, t), "a": _normal(g, (m, k), 1.0, t), "b": _weight(g, wide, k, t)[0]}
    if op == "gated_grad" or case["act"] != "none":
        d["z"] = _normal(g, (m, wide), 1.0, t)
    return d


def prepare(case, seed):
    state = {"case": case, "in": _inputs(case, seed)}
    if own:
        # what a training or serving loop keeps: the operator's handle and its result buffers
        op = _operator(case)
        state["launch"] = op.bind(*state["in"].values())
    return state


def _operator(case):
    import compiler_hlo_amd as H
    op, t = case["op"], case["dtype"]
    act = None if case.get("act", "none") == "none" else case["act"]
    if op == "norm":
        return H.RmsNorm(case["rows"], case["cols"], t, residual=case["residual"], out_dtype=case["out"], eps=EPS)
    if op == "norm_grad":
        return H.RmsNormGrad(case["rows"], case["cols"], t, stream_grad=case["residual"])
    if op == "dropout":
        return H.Dropout(case["rows"], case["cols"], t, p=case["p"], residual=case["residual"])
    m, n, k = case["m"], case["n"], case["k"]
    if op == "product":
        return H.Matmul(m, n, k, t, out_dtype=case["out"], bias=case["bias"], activation=act,
                        residual=case["residual"])
    if op == "product_grad":
        return H.MatmulGrad(m, n, k, t, bias=case["bias"], activation=act)
    if op == "gated":
        return H.GatedFeedForward(m, n, k, t, out_dtype=case["out"], activation=act, save=case["save"])
    return H.GatedFeedForwardGrad(m, n, k, t, activation=act)


# --------------------------------------------------------------------------
# one pass
# --------------------------------------------------------------------------
def run(state):
    if own:
        return state["launch"]()
    case, d = state["case"], state["in"]
    return {"norm": _norm, "norm_grad": _norm_grad, "product": _product, "product_grad": _product_grad,
            "gated": _gated, "gated_grad": _gated_grad, "dropout": _dropout}[case["op"]](case, **d)


def _norm(case, x, weight, residual=None):
    h = x.float()
    if residual is not None:
        h = h + residual.float()
    rstd = torch.rsqrt((h * h).mean(1) + EPS)
    y = h * rstd[:, None] * weight.float()
    stream = () if residual is None else (h.to(x.dtype),)
    if case["out"] not in QMAX:
        return (y.to(x.dtype), *stream, rstd)
    qmax = QMAX[case["out"]]
    scale = y.abs().amax(1) / qmax
    q = (y / torch.where(scale > 0, scale, 1.0)[:, None]).clamp(-qmax, qmax).to(TORCH[case["out"]])
    return (q, scale, *stream, rstd)


def _norm_grad(case, dy, h, weight, rstd, dstream=None):
    dy, x = dy.float(), h.float() * rstd[:, None]
    g = dy * weight.float()
    dx = (g - x * (g * x).mean(1, keepdim=True)) * rstd[:, None]
    if dstream is not None:
        dx = dx + dstream.float()
    return dx.to(h.dtype), (dy * x).sum(0)


def _sigmoid(z):
    return 1 / (1 + torch.exp(-z))


def _act(kind, z):
    """(act(z), act'(z))"""
    if kind == "relu":
        return torch.clamp(z, min=0), (z > 0).to(z.dtype)
    if kind == "silu":
        s = _sigmoid(z)
        return z * s, s * (1 + z * (1 - s))
    if kind == "gelu":
        c = math.sqrt(2 / math.pi)
        t = torch.tanh(c * (z + 0.044715 * z * z * z))
        return 0.5 * z * (1 + t), 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * c * (1 + 3 * 0.044715 * z * z)
    return z, torch.ones_like(z)


def _matmul(a, b, a_scale, b_scale):
    z = a.float() @ b.float().T
    return z if a_scale is None else z * a_scale[:, None] * b_scale


def _product(case, a, b, a_scale=None, b_scale=None, bias=None, residual=None):
    z = _matmul(a, b, a_scale, b_scale)
    if bias is not None:
        z = z + bias.float()
    y = _act(case["act"], z)[0]
    if residual is not None:
        y = y + residual.float()
    return y.to(TORCH[case["out"]])


def _product_grad(case, dd, a, b, z=None):
    dz = dd.float()
    if z is not None:
        dz = dz * _act(case["act"], z.float())[1]
    grads = (dz @ b.float()).to(a.dtype), (dz.T @ a.float()).to(b.dtype)
    return (*grads, dz.sum(0)) if case["bias"] else grads


def _gated(case, a, b, a_scale=None, b_scale=None):
    z = _matmul(a, b, a_scale, b_scale)
    gate, up = z[:, :case["n"]], z[:, case["n"]:]
    h = (_act(case["act"], gate)[0] * up).to(TORCH[case["out"]])
    return (h, z.to(TORCH[case["out"]])) if case["save"] else h


def _gated_grad(case, dd, a, b, z):
    dd, gate, up = dd.float(), z[:, :case["n"]].float(), z[:, case["n"]:].float()
    f, df = _act(case["act"], gate)
    dz = torch.cat([dd * up * df, dd * f], 1)
    return (dz @ b.float()).to(a.dtype), (dz.T @ a.float()).to(b.dtype)


LOW = 0xFFFFFFFF


def _mul32(m, x):
    """The high and the low 32 bits of m * x, 32-bit values held in int64."""
    lo, hi = m * (x & 0xFFFF), m * (x >> 16)
    mid = hi + (lo >> 16)
    return mid >> 16, ((mid & 0xFFFF) << 16) | (lo & 0xFFFF)


def _words(count, state):
    """Philox4x32-10 of the counters offset, offset + 1, ...: [count, 4] words in int64."""
    key0, key1 = state[0] & LOW, (state[0] >> 32) & LOW
    at = torch.arange(count, device=state.device) + state[1]
    a, b = at & LOW, (at >> 32) & LOW
    c, d = torch.zeros_like(a), torch.zeros_like(a)
    for i in range(10):
        h0, l0 = _mul32(0xD2511F53, a)
        h1, l1 = _mul32(0xCD9E8D57, c)
        a, b, c, d = h1 ^ b ^ ((key0 + i * 0x9E3779B9) & LOW), l1, h0 ^ d ^ ((key1 + i * 0xBB67AE85) & LOW), l0
    return torch.stack([a, b, c, d], 1)


def _dropout(case, x, state, residual=None):
    # 16 bits an element: the low half of a word, then its high half
    w = _words(-(-x.numel() // 8), state)
    bits = torch.stack([w & 0xFFFF, w >> 16], 2).reshape(-1)[:x.numel()].reshape(x.shape)
    cut = round(case["p"] * 65536)
    y = torch.where(bits >= cut, x.float() * (65536 / (65536 - cut)), 0.0)
    if residual is not None:
        y = y + residual.float()
    return y.to(x.dtype)


# --------------------------------------------------------------------------
# what a pass cannot do without
# --------------------------------------------------------------------------
def work(case):
    op, e = case["op"], BYTES[case["dtype"]]
    if op in ("norm", "norm_grad", "dropout"):
        rows, cols = case["rows"], case["cols"]
        size, more = rows * cols, 1 if case["residual"] else 0
        if op == "norm":
            out = BYTES[case["out"]]
            return {"bytes": size * (e * (1 + 2 * more) + out) + cols * e + rows * (8 if out == 1 else 4), "flops": 6 * size}
        if op == "norm_grad":
            return {"bytes": size * e * (3 + more) + cols * (e + 4) + rows * 4, "flops": 10 * size}
        return {"bytes": size * e * (2 + more) + 16, "flops": 2 * size}
    m, n, k = case["m"], case["n"], case["k"]
    wide = n if op.startswith("product") else 2 * n
    if op in ("product", "gated"):
        out = BYTES[case["out"]]
        extra = (m + wide) * 4 if e == 1 else 0
        extra += n * out if case.get("bias") else 0
        extra += m * n * out if case.get("residual") else 0
        extra += m * wide * out if case.get("save") else 0
        return {"bytes": (m * k + wide * k) * e + m * n * out + extra, "flops": 2 * m * wide * k}
    extra = m * wide * e if op == "gated_grad" or case["act"] != "none" else 0
    extra += n * 4 if case.get("bias") else 0
    return {"bytes": m * n * e + extra + 2 * (m * k + wide * k) * e, "flops": 4 * m * wide * k}


# --------------------------------------------------------------------------
# the definition, in 64 bits
# --------------------------------------------------------------------------
def _phi(kind, z):
    """The activation and its derivative from their definitions."""
    if kind == "none":
        return z, z * 0 + 1
    if kind == "relu":
        return z.relu(), (z > 0).double()
    if kind == "silu":
        e = z.sigmoid()
        return z * e, e + z * e * (1 - e)
    # GELU's tanh form as z * sigmoid(2u), u = sqrt(2/pi) (z + 0.044715 z^3)
    u = math.sqrt(2 / math.pi) * (z + 0.044715 * z.pow(3))
    e = (2 * u).sigmoid()
    return z * e, e + 2 * z * e * (1 - e) * math.sqrt(2 / math.pi) * (1 + 0.134145 * z.pow(2))


def _keeps(count, seed, offset, cut):
    """Which of `count` elements are kept, with numpy's unsigned 64-bit arithmetic."""
    u64, low = np.uint64, np.uint64(LOW)
    at = np.arange(-(-count // 8), dtype=u64) + u64(offset % 2**64)
    x = [at & low, at >> u64(32), np.zeros_like(at), np.zeros_like(at)]
    key = [seed & LOW, (seed >> 32) & LOW]
    for _ in range(10):
        p, q = x[0] * u64(0xD2511F53), x[2] * u64(0xCD9E8D57)
        x = [(q >> u64(32)) ^ x[1] ^ u64(key[0]), q & low, (p >> u64(32)) ^ x[3] ^ u64(key[1]), p & low]
        key = [(key[0] + 0x9E3779B9) & LOW, (key[1] + 0xBB67AE85) & LOW]
    halves = np.stack([x[0], x[1], x[2], x[3]], 1).astype("<u4").view("<u2").reshape(-1)[:count]
    return torch.from_numpy(halves >= cut).cuda()


def exact(case, seed):
    op = case["op"]
    d = {name: v if name == "state" else v.double() for name, v in _inputs(case, seed).items()}
    if op == "norm":
        h = d["x"] + d["residual"] if case["residual"] else d["x"]
        rms = (h.pow(2).sum(1) / case["cols"] + EPS).sqrt()
        y = h / rms[:, None] * d["weight"]
        stream = [h] if case["residual"] else []
        if case["out"] in QMAX:
            scale = y.abs().max(1).values / QMAX[case["out"]]
            return [y / scale[:, None], scale, *stream, 1 / rms]
        return [y, *stream, 1 / rms]
    if op == "norm_grad":
        # y_j = w_j h_j r with r = (mean h^2 + eps)^(-1/2): dr/dh_i = -r^3 h_i / cols
        r = d["rstd"][:, None]
        through = (d["dy"] * d["weight"] * d["h"]).sum(1, keepdim=True)
        dx = d["dy"] * d["weight"] * r - d["h"] * r.pow(3) * through / case["cols"]
        if case["residual"]:
            dx = dx + d["dstream"]
        return [dx, (d["dy"] * d["h"] * r).sum(0)]
    if op == "dropout":
        cut = round(case["p"] * 65536)
        seed_, offset = d["state"].tolist()
        keep = _keeps(d["x"].numel(), seed_, offset, cut).reshape(d["x"].shape)
        y = d["x"] * keep * 65536 / (65536 - cut)
        return y + d["residual"] if case["residual"] else y
    a, b, n = d["a"], d["b"], case["n"]
    if op in ("product", "gated"):
        if "a_scale" in d:
            a, b = a * d["a_scale"][:, None], b * d["b_scale"][:, None]
        z = torch.mm(a, b.t())
        if op == "gated":
            h = _phi(case["act"], z[:, :n])[0] * z[:, n:]
            return [h, z] if case["save"] else h
        if case["bias"]:
            z = z + d["bias"]
        y = _phi(case["act"], z)[0]
        return y + d["residual"] if case["residual"] else y
    if op == "product_grad":
        dz = d["dd"] * _phi(case["act"], d["z"])[1] if "z" in d else d["dd"]
        return [torch.mm(dz, b), torch.mm(dz.t(), a)] + ([dz.sum(0)] if case["bias"] else [])
    f, df = _phi(case["act"], d["z"][:, :n])
    dgate, dup = d["dd"] * d["z"][:, n:] * df, d["dd"] * f
    return [torch.mm(dgate, b[:n]) + torch.mm(dup, b[n:]),
            torch.cat([torch.mm(dgate.t(), a), torch.mm(dup.t(), a)])]
