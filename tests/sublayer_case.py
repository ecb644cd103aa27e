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


# ------------------------------------------------------- gated projections --
ACTS = ("silu", "gelu", "gelu_tanh", "relu")  # in the order of the MHC_ACT numbers


def act(g, name):
    """(activation, derivative, the argument of its exponential) in 64 bits."""
    g = g.double()
    if name == "relu":
        return torch.where(g > 0, g, 0.0), (g > 0).double(), torch.zeros_like(g)
    if name == "gelu":
        p = 0.5 * torch.erfc(-g / math.sqrt(2))
        return g * p, p + g * torch.exp(-g * g / 2) / math.sqrt(2 * math.pi), g * g / 2
    q = g if name == "silu" else math.sqrt(8 / math.pi) * (g + 0.044715 * g ** 3)
    dq = 1.0 if name == "silu" else math.sqrt(8 / math.pi) * (1 + 3 * 0.044715 * g ** 2)
    s = torch.sigmoid(q)
    return g * s, s + g * s * (1 - s) * dq, q


def glu(x, w, add, name):
    """{h, gu} and the sums of their terms' absolute values, in units of 2^-24 roundings.

    A sum of H products (exact in fp32) is off by at most 2 H 2^-24 of the products' absolute sum (H
    additions, each off by at most a whole unit: the tensor cores' rounding is not documented); the
    activation has a slope below 1.2, and its own error is some units and one per unit of the
    exponential's argument."""
    F = w.shape[0] // 2
    H = x.shape[1]
    gu, size = x.double() @ w.double().t(), x.double().abs() @ w.double().abs().t()
    if add is not None:
        gu, size = gu + add.double(), size + add.double().abs()
    g, u = gu[:, :F], gu[:, F:]
    a, _, q = act(g, name)
    off = 2 * (H + 1) * size
    terms = 1.2 * off[:, :F] * u.abs() + a.abs() * off[:, F:] + (64 + 4 * q.abs()) * (a * u).abs()
    # the product of both errors
    terms = terms + off[:, :F] * off[:, F:] * 2.0 ** -24
    return {"h": a * u, "gu": gu}, {"h": terms, "gu": off}


def glu_grad(dh, gu, x, w, name, dtype):
    """{dgu, dx, dw} and their terms in units of 2^-24: dgu's rounding to its type enters the products
    with at most half a unit of each factor, and their sums as in glu()."""
    from block_case import TINY, UNIT
    F = dh.shape[1]
    g, u, d = gu[:, :F].double(), gu[:, F:].double(), dh.double()
    a, da, q = act(g, name)
    dgu = torch.cat([d * u * da, d * a], 1)
    # the derivative is a sum of terms of up to |g| (1 + |q'|): some units of each, and one per unit of the exponential's argument
    slope = 1.0 if name in ("silu", "relu") else math.sqrt(8 / math.pi) * (1 + 3 * 0.044715 * g ** 2) if name == "gelu_tanh" else 1.0
    size = 1.2 + (g.abs() * slope * torch.exp(-q.abs()) if name != "gelu" else g.abs() * torch.exp(-q) * 0.4)
    n = 64 + 4 * q.abs()
    off = torch.cat([n * (d * u).abs() * size, n * (d * a).abs()], 1)
    step = (UNIT[dtype] * dgu.abs() * (1 + 2.0 ** -7) + TINY[dtype]) * 2.0 ** 24 + off
    out = {"dgu": dgu, "dx": dgu @ w.double(), "dw": dgu.t() @ x.double()}
    big = dgu.abs() + step * 2.0 ** -24
    return out, {"dgu": off, "dx": (step + 2 * (2 * F + 1) * big) @ w.double().abs(),
                 "dw": (step + 2 * (len(x) + 1) * big).t() @ x.double().abs()}


# --------------------------------------------------------------- adapters --
def lora(x, a, b, index, scale, base):
    """(out, its terms in units of 2^-24): v = A x is off by 2 H units of its products' absolute sum and, as two
    16-bit values of a row brought to at most 2, by 2^-16 of itself (bf16; both halves round to nearest) or
    2^-24 of the row's largest (fp16's subnormal step); B v by 2 R units of each of its two sums."""
    T, H = x.shape
    n, N, R = b.shape
    out, terms = torch.zeros(T, N, dtype=torch.float64), torch.zeros(T, N, dtype=torch.float64)
    if base is not None:
        out, terms = base.double().clone(), base.double().abs()
    for t in range(T):
        i = int(index[t])
        if not 0 <= i < n:
            continue
        s = 1.0 if scale is None else float(scale[i])
        A, Bm, X = a[i].double(), b[i].double(), x[t].double()
        v, size = A @ X, A.abs() @ X.abs()
        off = 2 * (H + 32) * size + 2.0 ** 8 * v.abs() + 4 * v.abs().max() + 2 * (2 * R + 4) * (v.abs() + size * (H + 32) * 2.0 ** -23)
        out[t] += s * (Bm @ v)
        terms[t] += abs(s) * (Bm.abs() @ off) + 4 * abs(s) * (Bm @ v).abs()
    return out, terms
