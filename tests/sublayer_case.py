"""Plain 64-bit implementations of the operators inside a block (CPU torch): the
gated projections and their gradient, adapters of many requests, dropout.
Tolerances are block_case.check's: half a unit of the output's type plus the fp32
roundings of the longest chain, on the sum of the terms' absolute values."""
from __future__ import annotations

import math

import torch

LOW = 0xFFFFFFFF


# ---------------------------------------------------------------- dropout --
def philox(counter, key):
    """Philox 4x32 with ten rounds on Python integers: four words of a counter of four, under a key of two."""
    a, b, c, d = counter
    k0, k1 = key
    for _ in range(10):
        p, q = a * 0xD2511F53, c * 0xCD9E8D57
        a, b, c, d = (q >> 32) ^ b ^ k0, q & LOW, (p >> 32) ^ d ^ k1, p & LOW
        k0, k1 = (k0 + 0x9E3779B9) & LOW, (k1 + 0xBB67AE85) & LOW
    return a, b, c, d


def words(T, H, key, call):
    """[T, H] words of a dropout call (int64)."""
    key, call = key % 2 ** 64, call % 2 ** 64
    w = []
    for i in range(T * H // 4):
        w += philox((i & LOW, i >> 32, call & LOW, call >> 32), (key & LOW, key >> 32))
    return torch.tensor(w, dtype=torch.int64).view(T, H)


def dropout(y, r, p, key, call):
    """(out, sum of absolute terms)."""
    keep = words(*y.shape, key, call) >= math.floor(p * 2 ** 32 + 0.5)
    x = torch.where(keep, y.double() / (1 - p) if p < 1 else 0.0, 0.0)
    return (x, x.abs()) if r is None else (x + r.double(), x.abs() + r.double().abs())
