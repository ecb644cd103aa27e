"""Whole-number inputs for the operators inside a block, and what they give bit for bit.

Every product and every sum of products below stays under 2^24, where fp32 holds whole numbers
exactly in whatever order they are added, so an output has ONE value: the exact number rounded once
to the output's type.  A sum that loses a single column of its reduction, or a part of it that was
kept in fewer bits, gives another one.  (The bounds of sublayer_case grow with the length of the sum
and cannot tell.)"""
from __future__ import annotations

import torch


def whole(g, *shape, most, dtype=torch.float32):
    return torch.randint(-most, most + 1, shape, generator=g).to(dtype)


# ------------------------------------------------------- gated projections --
GLU = [  # T, H, F: few tokens in runs, small and large tiles, tiles cut along H, remainders of H
    (1, 5120, 2048), (4, 2048, 5000), (9, 5120, 2000), (16, 16384, 520), (2, 72, 40000), (17, 5120, 1032), (24, 1024, 20000),
    (64, 5120, 1032), (130, 8192, 264), (129, 16384, 8), (128, 16384, 24), (256, 4096, 10000), (300, 2056, 136), (1003, 2048, 5000),
    (2304, 1536, 4224), (16384, 64, 72)]


def glu_inputs(T, H, F, dtype, device="cpu"):
    """x, w, add: sums of at most 64 H + 100 <= 2^20 + 100."""
    g = torch.Generator().manual_seed(T + H + F)
    return tuple(whole(g, *s, most=m, dtype=dtype).to(device) for s, m in (((T, H), 8), ((2 * F, H), 8), ((T, 2 * F), 100)))


def glu(x, w, add, dtype):
    """(h, gu) of max(g, 0) * u: g and u are exact, their product is rounded to fp32 and then to the type."""
    gu = x.double() @ w.double().t() + add.double()
    assert float(gu.abs().max()) < 2 ** 24
    F = gu.shape[1] // 2
    return (gu[:, :F].clamp_min(0).float() * gu[:, F:].float()).to(dtype), gu.to(dtype)


# --------------------------------------------------------- their gradient --
GRAD = [(3000, 520, 2000), (128, 512, 20000), (20000, 72, 64), (1024, 1024, 4096), (700, 2920, 1000), (5, 40, 16384),
        (1003, 512, 1368), (64, 256, 8192), (64, 512, 1368)]


def grad_inputs(T, H, F, dtype, device="cpu"):
    """dh, gu, x, w: dgu at most 16, so exact in every type; sums of at most 128 max(2F, T) < 2^24."""
    g = torch.Generator().manual_seed(T + H + F)
    sizes = (((T, F), 2), ((T, 2 * F), 8), ((T, H), 8), ((2 * F, H), 8))
    return tuple(whole(g, *s, most=m, dtype=dtype).to(device) for s, m in sizes)


def grad(dh, gu, x, w):
    """(dgu, dx, dw) of max(g, 0) * u, exact."""
    F = dh.shape[1]
    g, u, d = gu[:, :F].double(), gu[:, F:].double(), dh.double()
    dgu = torch.cat([d * u * (g > 0), d * g.clamp_min(0)], 1)
    dx, dw = dgu @ w.double(), dgu.t() @ x.double()
    assert max(float(dx.abs().max()), float(dw.abs().max())) < 2 ** 23
    return dgu, dx, dw


# --------------------------------------------------------------- adapters --
LORA = [  # T, H, N, R, n
    (1, 5120, 200, 16, 2), (64, 5120, 136, 64, 5), (40, 2056, 72, 256, 3), (65, 5120, 1000, 8, 3), (1003, 2048, 520, 24, 5),
    (1003, 2056, 520, 40, 70), (2100, 1032, 264, 64, 4), (700, 5120, 136, 128, 3), (1500, 520, 392, 256, 40), (300, 5120, 72, 192, 1)]


def lora_inputs(T, H, N, R, n, dtype, device="cpu"):
    """x, a, b, index, scale, base: A x at most 4 H < 2^15 (two 16-bit values hold 16 bits), scales 1 and 2."""
    g = torch.Generator().manual_seed(T + H + N + R)
    x, a, b, base = (whole(g, *s, most=m, dtype=dtype) for s, m in (((T, H), 4), ((n, R, H), 1), ((n, N, R), 2), ((T, N), 100)))
    index, scale = torch.randint(-1, n + 1, (T,), generator=g).int(), torch.randint(1, 3, (n,), generator=g).float()
    return tuple(t.to(device) for t in (x, a, b, index, scale, base))


def lora(x, a, b, index, scale, base):
    """base + scale B (A x), exact."""
    out = base.double().clone()
    for i in range(len(a)):
        t = torch.nonzero(index == i)[:, 0]
        v = x[t].double() @ a[i].double().t()
        assert not len(t) or float(v.abs().max()) < 2 ** 15
        out[t] += float(scale[i]) * (v @ b[i].double().t())
    assert float(out.abs().max()) < 2 ** 23
    return out
