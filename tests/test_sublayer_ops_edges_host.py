"""The whole-number cases of the operators inside a block can tell: a sum that loses one stage of 64 of its reduction,
or the last eight of it, and one with a part kept in 16 bits give other outputs (planted here in the oracle)."""
import pytest
import torch

import sublayer_exact_case as X

DTYPES = (torch.bfloat16, torch.float16)


def lose(t, dim, first, count):
    """`t` with `count` entries of its dimension `dim` from `first` on as zeros."""
    t = t.clone()
    t.narrow(dim, first, min(count, t.shape[dim] - first)).zero_()
    return t


def differs(a, b, dtype):
    return float((a.to(dtype) != b.to(dtype)).double().mean())


@pytest.mark.parametrize("T,H,F", X.GLU)
@pytest.mark.parametrize("dtype", DTYPES)
def test_projections_tell(T, H, F, dtype):
    x, w, add = X.glu_inputs(T, H, F, dtype)
    x, w, add = x[:40], w[:80], add[:40, :80]  # (some tokens and features)
    gu = X.glu(x, w, add, dtype)[1]
    for first, count in ((H // 2 // 64 * 64, 64), (H - 8, 8)):
        assert differs(gu, X.glu(lose(x, 1, first, count), w, add, dtype)[1], dtype) > 0.5
    if H >= 2048:  # long enough to be cut: half of the sum in 16 bits
        half = x[:, :H // 2].double() @ w[:, :H // 2].double().t()
        rest = x[:, H // 2:].double() @ w[:, H // 2:].double().t() + add.double()
        assert differs(gu, half.to(torch.bfloat16).double() + rest, dtype) > 0.05


@pytest.mark.parametrize("T,H,F", X.GRAD)
def test_gradient_tells(T, H, F):
    dh, gu, x, w = X.grad_inputs(T, H, F, torch.bfloat16)
    dgu = X.grad(dh, gu, x[:, :8], w[:, :8])[0]
    for first, count in ((T // 2 // 64 * 64, 64), (max(T - 8, 0), 8)):  # dw, as fp32: over the tokens
        a, x8 = dgu[:, :40], x[:, :40].double()
        assert differs(a.t() @ x8, a.t() @ lose(x8, 0, first, count), torch.float32) > 0.5
    for first, count in ((F // 64 * 64, 64), (2 * F - 8, 8)):  # dx, as bf16: over 2F
        a, w8 = dgu[:40], w[:, :40].double()
        assert differs(a @ w8, a @ lose(w8, 0, first, count), torch.bfloat16) > 0.3


@pytest.mark.parametrize("T,H,N,R,n", X.LORA)
def test_adapters_tell(T, H, N, R, n):
    x, a, b, index, scale, base = X.lora_inputs(T, H, N, R, n, torch.bfloat16)
    index = index.clamp(0, n - 1)[:40]
    x, base, b = x[:40], base[:40, :40], b[:, :40]
    out = X.lora(x, a, b, index, scale, base)
    for first, count in ((H // 2 // 64 * 64, 64), (H - 8, 8)):
        assert differs(out, X.lora(lose(x, 1, first, count), a, b, index, scale, base), torch.bfloat16) > 0.3
    assert differs(out, X.lora(x, lose(a, 1, R - 8, 8), b, index, scale, base), torch.bfloat16) > 0.3
