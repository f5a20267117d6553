"""The feed-forward layer by experts and its 8-bit products with block scales,
case by case: what each operator reads and writes, its plain form, and its
value from the definition.

Four operators, with their backward directions:

* ``route``    (token, choice) pairs sorted by expert, and the tokens' rows
               copied to the sorted places (with their scales in 8 bits);
* ``combine``  rows back in the tokens' order, d[t] = sum_j w[t, j]
               y[place[t, j]] + residual[t], and the gradient of y and w;
* ``experts``  every expert's product, plain or gated, over its rows of the
               sorted array, in 16 bits or in e4m3 with block scales, and the
               gradient of rows and weights;
* ``blocks``   e4m3 with a scale for each block of 128: rows quantised, and the
               product of such operands.

A pair whose expert lies outside 0 .. experts - 1 (another rank's) has place -1.
Scales of rows are [blocks, rows], those of weights [blocks of rows, blocks].
A case is a dict of plain values.  ``own`` chooses between the plain form and
the library's operators.
"""
import math

import numpy as np
import torch

own = False

TORCH = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16, "f8e4m3": torch.float8_e4m3fn}
BYTES = {"f32": 4, "bf16": 2, "f16": 2, "f8e4m3": 1}
TOP = 448.0
BLOCK = 128


# --------------------------------------------------------------------------
# cases
# --------------------------------------------------------------------------
def route(name, tokens, top_k, experts, cols, dtype, shard):
    return {"name": name, "op": "route", "tokens": tokens, "top_k": top_k, "experts": experts, "cols": cols,
            "dtype": dtype, "shard": shard}


def combine(name, tokens, top_k, experts, cols, dtype, residual, shard):
    return {"name": name, "op": "combine", "tokens": tokens, "top_k": top_k, "experts": experts, "cols": cols,
            "dtype": dtype, "residual": residual, "shard": shard}


def combine_grad(name, tokens, top_k, experts, cols, dtype, shard):
    return {"name": name, "op": "combine_grad", "tokens": tokens, "top_k": top_k, "experts": experts, "cols": cols,
            "dtype": dtype, "shard": shard}


def experts(name, tokens, top_k, count, n, k, dtype, gated, shard):
    return {"name": name, "op": "experts", "tokens": tokens, "top_k": top_k, "experts": count, "n": n, "k": k,
            "dtype": dtype, "gated": gated, "shard": shard}


def experts_grad(name, tokens, top_k, count, n, k, dtype, gated, shard):
    return experts(name, tokens, top_k, count, n, k, dtype, gated, shard) | {"op": "experts_grad"}


def quantize(name, rows, cols, dtype):
    return {"name": name, "op": "quantize", "rows": rows, "cols": cols, "dtype": dtype}


def blocks(name, m, n, k, out, gated, residual):
    return {"name": name, "op": "blocks", "m": m, "n": n, "k": k, "out": out, "gated": gated, "residual": residual}


def listed():
    return [
        # a decode step's tokens sorted by expert: launch latency
        route("route_decode_bf16", 24, 8, 128, 4096, "bf16", False),
        # a long prompt's rows, already in 8 bits, sent to a rank that holds half of the experts
        route("route_prompt_f8", 8191, 8, 64, 4096, "f8e4m3", True),
        # a single token's expert rows summed up: the shortest call of a decode step
        combine("combine_token_f16", 1, 8, 64, 4096, "f16", False, False),
        # a prompt's expert rows summed up and added to the residual stream
        combine("combine_prompt_bf16", 4099, 8, 64, 4096, "bf16", True, False),
        # the sum's backward pass in a training step
        combine_grad("combine_backward_bf16", 8192, 4, 32, 4096, "bf16", False),
        # gate and up projections of a decode batch, a few rows an expert: bound by the experts' weights
        experts("experts_decode_f8", 32, 4, 32, 1408, 4096, "f8e4m3", True, False),
        # gate and up projections of a prompt, odd number of tokens
        experts("experts_prompt_bf16", 4099, 2, 8, 4096, 4096, "bf16", True, False),
        # the gradient of a down projection by experts in a training step
        experts_grad("experts_backward_bf16", 8192, 2, 16, 4096, 1408, "bf16", False, False),
        # one token's row quantised for the next product
        quantize("quantize_token_bf16", 1, 11264, "bf16"),
        # a prompt's rows quantised
        quantize("quantize_prompt_bf16", 8191, 11264, "bf16"),
        # the down projection of a single token, added to the residual stream: bound by the weights
        blocks("blocks_token_f8", 1, 4096, 16384, "bf16", False, True),
        # the down projection of a prompt
        blocks("blocks_prompt_f8", 4099, 4096, 16384, "bf16", False, True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _dims(rng, lo, hi, step):
    return step * max(1, _log(rng, lo, hi) // step)


def draw(rng):
    op = rng.choice(["route", "combine", "combine_grad", "experts", "experts", "experts_grad", "quantize", "blocks"])
    half = rng.choice(["bf16", "bf16", "f16"])
    step = rng.choice([64, 64, 64, 8, 1])
    if op == "quantize":
        cols = _dims(rng, 64, 16384, rng.choice([128, 128, 8, 1]))
        rows = min(_log(rng, 1, 16384), 8191 * 11264 // cols)
        return quantize("drawn", rows, cols, rng.choice([half, half, "f32"]))
    if op == "blocks":
        m, n, k = _log(rng, 1, 8192), _dims(rng, 256, 11264, step), _dims(rng, 256, 16384, step)
        gated = rng.random() < 0.5
        k = max(256, min(k, 4099 * 4096 * 16384 // (m * n * (1 + gated))))
        return blocks("drawn", m, n, k, half, gated, not gated and rng.random() < 0.5)
    count, shard = _log(rng, 1, 256), rng.random() < 0.25
    top_k = rng.randint(1, min(8, count))
    if op in ("route", "combine", "combine_grad"):
        cols = _log(rng, 64, 16384)
        if rng.random() < 0.7:
            cols = 16 * max(4, cols // 16)
        tokens = max(1, min(_log(rng, 1, 16384), 8191 * 8 * 2048 // (top_k * cols)))
        if op == "route":
            return route("drawn", tokens, top_k, count, cols, rng.choice([half, half, "f32", "f8e4m3"]), shard)
        dtype = rng.choice([half, half, half, "f32"])
        if op == "combine":
            return combine("drawn", tokens, top_k, count, cols, dtype, rng.random() < 0.5, shard)
        return combine_grad("drawn", tokens, top_k, count, cols, dtype, shard)
    # token counts of every size; features mostly in steps of 64, sometimes odd
    gated = rng.random() < 0.5
    n, k = _dims(rng, 128, 4096, step), _dims(rng, 128, 4096, step)
    count = max(1, min(count, 8 * 8192 * 4096 // ((1 + gated) * n * k)))
    top_k = min(top_k, count)
    tokens = max(1, min(_log(rng, 1, 8192), 8198 // top_k))
    if op == "experts":
        return experts("drawn", tokens, top_k, count, n, k, rng.choice([half, half, "f8e4m3"]), gated, shard)
    return experts_grad("drawn", tokens, top_k, count, n, k, half, gated, shard)


# --------------------------------------------------------------------------
# inputs
# --------------------------------------------------------------------------
def _normal(gen, shape, sigma, dtype):
    return (torch.randn(shape, generator=gen, device="cuda") * sigma).to(TORCH[dtype])


def _chosen(gen, case):
    """A router's choices, some experts liked more than others: ids and weights.
    A shard holds the middle half of twice as many experts."""
    count = case["experts"]
    every = 2 * count if case["shard"] else count
    score = torch.randn((case["tokens"], every), generator=gen, device="cuda")
    score += 0.5 * torch.randn(every, generator=gen, device="cuda")
    value, ids = score.topk(case["top_k"], 1)
    return (ids - (every - count) // 2).to(torch.int32), torch.softmax(value, 1)


def _sorted(ids, count):
    """(place, order, offsets) of a stable sort by expert."""
    flat = ids.reshape(-1).long()
    key = torch.where((flat >= 0) & (flat < count), flat, count)
    by = torch.argsort(key, stable=True)
    place = torch.empty_like(by)
    place[by] = torch.arange(by.numel(), device=by.device)
    place = torch.where(key < count, place, -1)
    order = torch.where(key[by] < count, by, -1)
    offsets = (key[None, :] < torch.arange(count + 1, device=by.device)[:, None]).sum(1)
    return place.reshape(ids.shape).to(torch.int32), order.to(torch.int32), offsets.to(torch.int32)


def _blocks_of(x):
    """Rows in e4m3 with a scale for each block of 128 of a row: y, scale [blocks, rows]."""
    rows, cols = x.shape
    count = -(-cols // BLOCK)
    wide = torch.nn.functional.pad(x.float(), (0, count * BLOCK - cols)).reshape(rows, count, BLOCK)
    scale = wide.abs().amax(2) / TOP
    y = (wide / torch.where(scale > 0, scale, 1.0)[:, :, None]).clamp(-TOP, TOP).to(TORCH["f8e4m3"])
    return y.reshape(rows, -1)[:, :cols].contiguous(), scale.T.contiguous()


def _weight_blocks(gen, parts, n, k):
    """`parts` weights of n rows (N(0, 1/k)), one after another, in e4m3 with a
    scale for each block of 128 x 128 of a part."""
    y = torch.empty((parts * n, k), dtype=TORCH["f8e4m3"], device="cuda")
    high, wide = -(-n // BLOCK), -(-k // BLOCK)
    scale = torch.empty((parts * high, wide), device="cuda")
    for p in range(parts):
        w = torch.randn((n, k), generator=gen, device="cuda") / math.sqrt(k)
        w = torch.nn.functional.pad(w, (0, wide * BLOCK - k, 0, high * BLOCK - n)).reshape(high, BLOCK, wide, BLOCK)
        s = w.abs().amax((1, 3)) / TOP
        w = (w / s[:, None, :, None]).clamp(-TOP, TOP).reshape(high * BLOCK, wide * BLOCK)
        y[p * n:(p + 1) * n] = w[:n, :k].to(TORCH["f8e4m3"])
        scale[p * high:(p + 1) * high] = s
    return y, scale


def _inputs(case, seed):
    """The inputs of a case by name, in the order in which the operator takes them."""
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    op, t = case["op"], case.get("dtype")
    if op == "quantize":
        # activations: some rows and columns larger than others
        x = torch.randn((case["rows"], case["cols"]), generator=g, device="cuda")
        x *= torch.exp(0.5 * torch.randn(case["cols"], generator=g, device="cuda"))
        return {"x": x.to(TORCH[t])}
    if op == "blocks":
        m, n, k = case["m"], case["n"], case["k"]
        a, sa = _blocks_of(torch.randn((m, k), generator=g, device="cuda"))
        b, sb = _weight_blocks(g, 2 if case["gated"] else 1, n, k)
        d = {"a": a, "b": b, "a_scale": sa, "b_scale": sb}
        if case["residual"]:
            d["residual"] = _normal(g, (m, n), 2.0, case["out"])
        return d
    ids, weight = _chosen(g, case)
    pairs = ids.numel()
    if op == "route":
        x = torch.randn((case["tokens"], case["cols"]), generator=g, device="cuda")
        if t == "f8e4m3":
            y, scale = _blocks_of(x)
            return {"expert": ids, "x": y, "x_scale": scale}
        return {"expert": ids, "x": x.to(TORCH[t])}
    place, _, offsets = _sorted(ids, case["experts"])
    if op in ("combine", "combine_grad"):
        shape = (case["tokens"], case["cols"])
        d = {"dd": _normal(g, shape, 0.02, t)} if op == "combine_grad" else {}
        d |= {"y": _normal(g, (pairs, case["cols"]), 1.0, t), "place": place, "weight": weight}
        if case.get("residual"):
            d["residual"] = _normal(g, shape, 2.0, t)
        return d
    n, k, count = case["n"], case["k"], case["experts"]
    parts = 2 if case["gated"] else 1
    if op == "experts":
        if t == "f8e4m3":
            a, sa = _blocks_of(torch.randn((pairs, k), generator=g, device="cuda"))
            b, sb = _weight_blocks(g, count * parts, n, k)
            return {"a": a, "b": b, "a_scale": sa, "b_scale": sb, "offsets": offsets}
        return {"a": _normal(g, (pairs, k), 1.0, t), "b": _normal(g, (count * parts * n, k), 1 / math.sqrt(k), t),
                "offsets": offsets}
    d = {"dd": _normal(g, (pairs, n), 0.02, t), "a": _normal(g, (pairs, k), 1.0, t),
         "b": _normal(g, (count * parts * n, k), 1 / math.sqrt(k), t)}
    if case["gated"]:
        d["z"] = _normal(g, (pairs, 2 * n), 1.0, t)
    return d | {"offsets": offsets}


def prepare(case, seed):
    state = {"case": case, "in": _inputs(case, seed)}
    if "offsets" in state["in"]:
        # what a program without an operator by experts has to know on the host
        state["ends"] = state["in"]["offsets"].tolist()
    if own:
        state["launch"] = _bound(case, **state["in"])
    return state


def _bound(case, **d):
    """What a training or serving loop keeps: the operators' handles and their
    result buffers.  Rows past the last expert's are left as they were: zeros."""
    import compiler_hlo_amd as H
    op, t = case["op"], case.get("dtype")

    def bind(o, *params):
        out = [torch.zeros(b.dims, dtype=_result(b.dtype), device="cuda") for b in o.results]
        return o.bind(*params, out=out)

    if op == "route":
        shape = (case["tokens"], case["top_k"])
        sort = bind(H.ExpertSort(*shape, case["experts"]), d["expert"])
        place = sort.results[0]
        if t == "f8e4m3":
            return sort, bind(H.ExpertDispatch(*shape, case["cols"], t, scales="blocks"), d["x"], place, d["x_scale"])
        return sort, bind(H.ExpertDispatch(*shape, case["cols"], t), d["x"], place)
    if op == "combine":
        o = H.ExpertCombine(case["tokens"], case["top_k"], case["cols"], t, residual=case["residual"])
    elif op == "combine_grad":
        o = H.ExpertCombineGrad(case["tokens"], case["top_k"], case["cols"], t)
    elif op == "quantize":
        o = H.BlockQuantize(case["rows"], case["cols"], t)
    elif op == "blocks":
        kind = H.GatedFeedForward if case["gated"] else H.Matmul
        more = {} if case["gated"] else {"residual": case["residual"]}
        o = kind(case["m"], case["n"], case["k"], "f8e4m3", out_dtype=case["out"], scales="blocks", **more)
    else:
        size = (case["tokens"] * case["top_k"], case["n"], case["k"])
        if op == "experts":
            kind = H.GatedFeedForward if case["gated"] else H.Matmul
            more = {"scales": "blocks", "out_dtype": "bf16"} if t == "f8e4m3" else {}
        else:
            kind, more = H.GatedFeedForwardGrad if case["gated"] else H.MatmulGrad, {}
        o = kind(*size, t, experts=case["experts"], **more)
    return (bind(o, *d.values()),)


def _result(dtype):
    return torch.int32 if dtype == "s32" else TORCH[dtype]


# --------------------------------------------------------------------------
# one pass
# --------------------------------------------------------------------------
def run(state):
    if own:
        out = []
        for launch in state["launch"]:
            r = launch()
            out += [r] if isinstance(r, torch.Tensor) else r
        return out
    case, d = state["case"], state["in"]
    more = {"ends": state["ends"]} if "ends" in state else {}
    out = {"route": _route, "combine": _combine, "combine_grad": _combine_grad, "experts": _experts,
           "experts_grad": _experts_grad, "quantize": _quantize, "blocks": _blocks}[case["op"]](case, **d, **more)
    return [out] if isinstance(out, torch.Tensor) else list(out)


def _route(case, expert, x, x_scale=None):
    place, order, offsets = _sorted(expert, case["experts"])
    token = torch.div(order.clamp(min=0), case["top_k"], rounding_mode="floor").long()
    bits = x.view(torch.uint8) if x_scale is not None else x
    y = torch.where((order >= 0)[:, None], bits[token], 0).view(x.dtype)
    if x_scale is None:
        return place, order, offsets, y
    return place, order, offsets, y, torch.where(order >= 0, x_scale[:, token], 0.0)


def _rows(y, place):
    """The rows at `place`, zeros at -1: [tokens, top_k, cols] in f32."""
    return torch.where((place >= 0)[:, :, None], y[place.clamp(min=0).long()].float(), 0.0)


def _combine(case, y, place, weight, residual=None):
    d = (_rows(y, place) * torch.where(place >= 0, weight, 0.0)[:, :, None]).sum(1)
    if residual is not None:
        d = d + residual.float()
    return d.to(y.dtype)


def _combine_grad(case, dd, y, place, weight):
    dd = dd.float()
    dweight = (_rows(y, place) * dd[:, None, :]).sum(2)
    pairs = y.shape[0]
    dy = torch.zeros((pairs + 1, y.shape[1]), device=y.device)  # one row more for what has no place
    at = torch.where(place >= 0, place, pairs).long().reshape(-1)
    dy[at] = (weight[:, :, None] * dd[:, None, :]).reshape(pairs, -1)
    return dy[:pairs].to(y.dtype), dweight


def _wide_rows(y, scale):
    """Rows in e4m3 with scales [blocks, rows], in f32."""
    return y.float() * scale.T.repeat_interleave(BLOCK, 1)[:, :y.shape[1]]


def _wide_weight(y, scale):
    """A weight in e4m3 with a scale for each block of 128 x 128, in f32."""
    n, k = y.shape
    return y.float() * scale.repeat_interleave(BLOCK, 0)[:n].repeat_interleave(BLOCK, 1)[:, :k]


def _silu(z):
    """(silu(z), its derivative)"""
    s = 1 / (1 + torch.exp(-z))
    return z * s, s * (1 + z * (1 - s))


# The experts' products go expert by expert, as a program does that has only
# matrix products of one weight.
def _experts(case, a, b, offsets, ends, a_scale=None, b_scale=None):
    n, parts = case["n"], 2 if case["gated"] else 1
    d = torch.zeros((a.shape[0], n), dtype=torch.bfloat16 if a_scale is not None else a.dtype, device=a.device)
    wide = _wide_rows(a, a_scale) if a_scale is not None else a.float()
    high = -(-n // BLOCK)
    for e, (lo, hi) in enumerate(zip(ends[:-1], ends[1:])):
        if lo == hi:
            continue
        z = []
        for p in range(e * parts, (e + 1) * parts):
            w = b[p * n:(p + 1) * n]
            w = w.float() if b_scale is None else _wide_weight(w, b_scale[p * high:(p + 1) * high])
            z.append(wide[lo:hi] @ w.T)
        d[lo:hi] = (_silu(z[0])[0] * z[1] if case["gated"] else z[0]).to(d.dtype)
    return d


def _experts_grad(case, dd, a, b, offsets, ends, z=None):
    n, parts = case["n"], 2 if case["gated"] else 1
    dz = dd.float()
    if z is not None:
        gate, up = z[:, :n].float(), z[:, n:].float()
        f, df = _silu(gate)
        dz = torch.cat([dz * up * df, dz * f], 1)
    da, db = torch.zeros_like(a), torch.zeros_like(b)
    for e, (lo, hi) in enumerate(zip(ends[:-1], ends[1:])):
        if lo < hi:
            rows = slice(e * parts * n, (e + 1) * parts * n)
            da[lo:hi] = (dz[lo:hi] @ b[rows].float()).to(a.dtype)
            db[rows] = (dz[lo:hi].T @ a[lo:hi].float()).to(b.dtype)
    return da, db


def _quantize(case, x):
    return _blocks_of(x)


def _blocks(case, a, b, a_scale, b_scale, residual=None):
    n, wide = case["n"], _wide_rows(a, a_scale)
    high = -(-n // BLOCK)
    z = wide @ _wide_weight(b[:n], b_scale[:high]).T
    if case["gated"]:
        z = _silu(z)[0] * (wide @ _wide_weight(b[n:], b_scale[high:]).T)
    if residual is not None:
        z = z + residual.float()
    return z.to(TORCH[case["out"]])


# --------------------------------------------------------------------------
# what a pass cannot do without
# --------------------------------------------------------------------------
def work(case):
    op = case["op"]
    if op == "quantize":
        size = case["rows"] * case["cols"]
        return {"bytes": size * (BYTES[case["dtype"]] + 1) + case["rows"] * -(-case["cols"] // BLOCK) * 4, "flops": 3 * size}
    if op == "blocks":
        m, n, k, e = case["m"], case["n"], case["k"], BYTES[case["out"]]
        parts, wide = 2 if case["gated"] else 1, -(-case["k"] // BLOCK)
        scales = 4 * wide * (m + parts * -(-n // BLOCK))
        return {"bytes": (m + parts * n) * k + scales + m * n * e * (2 if case["residual"] else 1),
                "flops": 2 * m * parts * n * k}
    t, pairs, count, e = case["tokens"], case["tokens"] * case["top_k"], case["experts"], BYTES[case["dtype"]]
    rows = pairs // 2 if case["shard"] else pairs  # that this shard has, about
    if op in ("route", "combine", "combine_grad"):
        cols = case["cols"]
        row = cols * e + (4 * -(-cols // BLOCK) if e == 1 else 0)
        if op == "route":
            return {"bytes": (t + rows) * row + 12 * pairs + 4 * count, "flops": 0}
        if op == "combine":
            return {"bytes": (rows + t * (2 if case["residual"] else 1)) * row + 8 * pairs, "flops": 2 * rows * cols}
        return {"bytes": (2 * rows + t) * row + 12 * pairs, "flops": 3 * rows * cols}
    n, k, parts = case["n"], case["k"], 2 if case["gated"] else 1
    # the experts that have a row, if all are liked alike
    used = count * (1 - (1 - min(1.0, rows / (t * count))) ** t)
    if op == "experts":
        out, scales = (2, 4 * -(-k // BLOCK) * (rows + used * parts * -(-n // BLOCK))) if e == 1 else (e, 0)
        return {"bytes": (rows + used * parts * n) * k * e + rows * n * out + scales, "flops": 2 * rows * parts * n * k}
    extra = rows * 2 * n * e if case["gated"] else 0
    return {"bytes": (rows * n + 2 * rows * k + (used + count) * parts * n * k) * e + extra,
            "flops": 4 * rows * parts * n * k}


# --------------------------------------------------------------------------
# the definition, in 64 bits
# --------------------------------------------------------------------------
def _spread(scale, cols):
    """Rows' scales for each of their elements."""
    return scale.double().t()[:, torch.arange(cols, device=scale.device) // BLOCK]


def _spread_weight(scale, n, k):
    """A weight's scales for each of its n x k elements."""
    at = [torch.arange(v, device=scale.device) // BLOCK for v in (n, k)]
    return scale.double()[at[0]][:, at[1]]


def exact(case, seed):
    op, d = case["op"], _inputs(case, seed)
    if op == "quantize":
        x = d["x"].double()
        cols = x.shape[1]
        scale = torch.stack([x[:, c:c + BLOCK].abs().max(1).values for c in range(0, cols, BLOCK)], 1) / TOP
        return [x / scale[:, torch.arange(cols, device=x.device) // BLOCK], scale.t()]
    if op == "blocks":
        m, n, k = case["m"], case["n"], case["k"]
        a = d["a"].double() * _spread(d["a_scale"], k)
        half = d["b_scale"].shape[0] // (2 if case["gated"] else 1)
        z = [torch.mm(a, (d["b"][i * n:(i + 1) * n].double() * _spread_weight(d["b_scale"][i * half:(i + 1) * half], n, k)).t())
             for i in range(2 if case["gated"] else 1)]
        y = z[0] * z[0].sigmoid() * z[1] if case["gated"] else z[0]
        return [y + d["residual"].double() if case["residual"] else y]
    if op == "route":
        ids, count, top_k = d["expert"].cpu().numpy().reshape(-1), case["experts"], case["top_k"]
        here = np.nonzero((ids >= 0) & (ids < count))[0]
        by = here[np.argsort(ids[here], kind="stable")]
        place, order = np.full(ids.size, -1), np.full(ids.size, -1)
        place[by] = np.arange(by.size)
        order[:by.size] = by
        offsets = np.concatenate([[0], np.cumsum(np.bincount(ids[here], minlength=count))])
        token = torch.from_numpy(by // top_k).cuda()
        x = d["x"].double()
        y = torch.zeros((ids.size, case["cols"]), dtype=torch.float64, device="cuda")
        y[:by.size] = x[token]
        out = [torch.from_numpy(v.astype(np.int32)).cuda() for v in (place.reshape(-1, top_k), order, offsets)] + [y]
        if "x_scale" in d:
            s = torch.zeros((d["x_scale"].shape[0], ids.size), dtype=torch.float64, device="cuda")
            s[:, :by.size] = d["x_scale"].double()[:, token]
            out.append(s)
        return out
    if op in ("combine", "combine_grad"):
        place, w, y = d["place"].long(), d["weight"].double(), d["y"]
        total = torch.zeros((case["tokens"], case["cols"]), dtype=torch.float64, device="cuda")
        dy = torch.zeros(y.shape, dtype=torch.float64, device="cuda") if op == "combine_grad" else None
        dw = torch.zeros_like(w)
        for j in range(case["top_k"]):
            has = (place[:, j] >= 0).nonzero()[:, 0]
            at = place[has, j]
            if op == "combine":
                total[has] += w[has, j, None] * y[at].double()
            else:
                up = d["dd"].double()[has]
                dy[at] = w[has, j, None] * up
                dw[has, j] = torch.linalg.vecdot(up, y[at].double())
        if op == "combine_grad":
            return [dy, dw]
        return [total + d["residual"].double() if case["residual"] else total]
    n, k, parts = case["n"], case["k"], 2 if case["gated"] else 1
    ends = d["offsets"].tolist()
    rows = d["a"].shape[0]
    a = d["a"].double()
    if "a_scale" in d:
        a = a * _spread(d["a_scale"], k)
    if op == "experts":
        out = torch.zeros((rows, n), dtype=torch.float64, device="cuda")
        for e in range(case["experts"]):
            at = slice(ends[e], ends[e + 1])
            if ends[e] == ends[e + 1]:
                continue
            z = []
            for p in range(parts * e, parts * (e + 1)):
                w = d["b"][p * n:(p + 1) * n].double()
                if "b_scale" in d:
                    high = -(-n // BLOCK)
                    w = w * _spread_weight(d["b_scale"][p * high:(p + 1) * high], n, k)
                z.append(torch.mm(a[at], w.t()))
            out[at] = z[0] * z[0].sigmoid() * z[1] if case["gated"] else z[0]
        return [out]
    dd = d["dd"].double()
    if case["gated"]:
        g, u = d["z"].double().chunk(2, 1)
        s = g.sigmoid()
        dd = torch.cat([dd * u * (s + g * s * (1 - s)), dd * g * s], 1)
    da = torch.zeros((rows, k), dtype=torch.float64, device="cuda")
    db = torch.zeros((case["experts"] * parts * n, k), dtype=torch.float64, device="cuda")
    for e in range(case["experts"]):
        at, to = slice(ends[e], ends[e + 1]), slice(e * parts * n, (e + 1) * parts * n)
        da[at] = torch.mm(dd[at], d["b"][to].double())
        db[to] = torch.mm(dd[at].t(), a[at])
    return [da, db]
