"""Plain forms of the operators in 64 bits, on the CPU, and the bounds of the
kernels' errors (test infrastructure).  Shares no code with the library."""
from __future__ import annotations

import math

import numpy as np
import torch

HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11,
        torch.float8_e4m3fn: 2.0 ** -4}
# half the spacing of the smallest numbers
TINY = {torch.float32: 2.0 ** -150, torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25,
        torch.float8_e4m3fn: 2.0 ** -10}


def f64(t):
    return t.detach().cpu().to(torch.float64)


def act(kind, z):
    """(act(z), act'(z)) from the definitions."""
    if kind is None:
        return z, torch.ones_like(z)
    if kind == "relu":
        return z.clamp(min=0), (z > 0).double()
    if kind == "silu":
        s = torch.sigmoid(z)
        return z * s, s * (1 + z * (1 - s))
    c = math.sqrt(2 / math.pi)
    t = torch.tanh(c * (z + 0.044715 * z ** 3))
    return 0.5 * z * (1 + t), 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * c * (1 + 3 * 0.044715 * z * z)


def act_error(z):
    """How far the kernel's act(z) and act'(z) may be off: the sigmoid's
    argument 2u carries a few roundings, so the sigmoid is off by that many
    units times its slope's argument; both functions grow no faster than |z|.
    |z| (|z| + 8) 2^-22 covers silu; GELU's argument is cubic, but where it is
    above 40 the sigmoid is 0 or 1 to 2^-57, which bounds it by 40."""
    a = z.abs()
    return (1 + a) * (torch.clamp(1.6 * a * (1 + 0.05 * a * a), max=40) + 8) * 2.0 ** -22


def sum_error(terms_abs, k):
    """k products added in 32 bits, in any order: k roundings (two units each:
    the matrix instructions' internal adds are taken at twice an IEEE add's
    error) of at most the sum of magnitudes."""
    return (k + 8) * 2.0 ** -23 * terms_abs


def close(got, want, error, dtype):
    """|got - want| <= one rounding of the result's type + `error`; a value
    that rounds past the type's largest number is an infinity."""
    got = f64(got)
    over = want.abs() >= torch.finfo(dtype).max * (1 + HALF[dtype])
    assert torch.equal(got[over], torch.sign(want[over]) * math.inf)
    got, want, error = got[~over], want[~over], (error[~over] if torch.is_tensor(error) else error)
    bound = HALF[dtype] * want.abs() * (1 + 2.0 ** -7) + TINY[dtype] + error
    bad = ~((got - want).abs() <= bound)
    assert not bad.any(), "%d of %d beyond the bound; worst %.3g of it; first at %s: got %r, want %r" % (
        int(bad.sum()), bad.numel(), float(((got - want).abs() / bound).max()),
        bad.nonzero()[0].tolist(), float(got[bad][0]), float(want[bad][0]))


def philox(counter, key):
    """Philox4x32-10 words [count, 4] of 64-bit counters (numpy uint64)."""
    m, low = (np.uint64(0xD2511F53), np.uint64(0xCD9E8D57)), np.uint64(0xFFFFFFFF)
    c = [counter & low, counter >> np.uint64(32), np.zeros_like(counter), np.zeros_like(counter)]
    k = [key & 0xFFFFFFFF, (key >> 32) & 0xFFFFFFFF]
    for _ in range(10):
        p, q = c[0] * m[0], c[2] * m[1]
        c = [(q >> np.uint64(32)) ^ c[1] ^ np.uint64(k[0]), q & low,
             (p >> np.uint64(32)) ^ c[3] ^ np.uint64(k[1]), p & low]
        k = [(k[0] + 0x9E3779B9) & 0xFFFFFFFF, (k[1] + 0xBB67AE85) & 0xFFFFFFFF]
    return np.stack(c, 1)


def keep_mask(count, seed, offset, p, first=0):
    """Elements first .. first + count - 1 (first a multiple of 8)."""
    at = (np.arange(first // 8, first // 8 + -(-count // 8), dtype=np.uint64) + np.uint64(offset % 2 ** 64))
    w = philox(at, seed % 2 ** 64)
    bits = np.stack([w & np.uint64(0xFFFF), w >> np.uint64(16)], 2).reshape(-1)[:count]
    cut = round(p * 65536)
    return torch.from_numpy(bits >= np.uint64(cut)), 65536 / (65536 - cut)
