"""Plain forms of the operators by expert and of block scales in 64 bits, on
the CPU (test infrastructure).  Shares no code with the library."""
from __future__ import annotations

import numpy as np
import torch

import operators_reference as R

F8 = torch.float8_e4m3fn


def sort(expert, experts):
    """(place, order, offsets) by a stable sort, in numpy."""
    ids = expert.cpu().numpy().reshape(-1).astype(np.int64)
    here = np.nonzero((ids >= 0) & (ids < experts))[0]
    by = here[np.argsort(ids[here], kind="stable")]
    place, order = np.full(ids.size, -1, np.int32), np.full(ids.size, -1, np.int32)
    place[by] = np.arange(by.size)
    order[:by.size] = by
    offsets = np.concatenate([[0], np.cumsum(np.bincount(ids[here], minlength=experts))]).astype(np.int32)
    return [torch.from_numpy(v) for v in (place.reshape(tuple(expert.shape)), order, offsets)]


def quantize(x):
    """Rows (f64) in e4m3 with a scale a block of 128, as BlockQuantize lays them out."""
    rows, cols = x.shape
    scale = torch.stack([x[:, c:c + 128].abs().amax(1) for c in range(0, cols, 128)]) / 448 if cols else x.new_zeros((0, rows))
    scale = scale.float()
    s = spread_rows(scale, cols)
    return (x / torch.where(s > 0, s, 1.0)).clamp(-448, 448).float().to(F8), scale


def quantize_weight(w):
    """A weight (f64) in e4m3 with a scale for each block of 128 x 128."""
    n, k = w.shape
    scale = torch.zeros((-(-n // 128), -(-k // 128)))
    for i in range(scale.shape[0]):
        for j in range(scale.shape[1]):
            scale[i, j] = float(w[i * 128:(i + 1) * 128, j * 128:(j + 1) * 128].abs().max()) / 448
    s = spread_weight(scale, n, k)
    return (w / torch.where(s > 0, s, 1.0)).clamp(-448, 448).float().to(F8), scale


def spread_rows(scale, cols):
    """[blocks, rows] as a factor for each element of [rows, cols]."""
    return R.f64(scale).T.repeat_interleave(128, 1)[:, :cols]


def spread_weight(scale, n, k):
    return R.f64(scale).repeat_interleave(128, 0)[:n].repeat_interleave(128, 1)[:, :k]
