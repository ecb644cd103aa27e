"""Refusals of the operators inside a block, and checks of their 64-bit test
implementations, without a GPU.  The addresses below are fake; every call
fails its checks before anything touches them."""
import math

import pytest
import torch

from mhc_residual_seam_gb300 import binding as B

import sublayer_case as R

A = 0x10000000  # 256-byte aligned, never dereferenced
STEP = 0x1000000


@pytest.fixture(scope="module")
def L():
    return B.lib()


def _call(fn, base, over):
    a = dict(base)
    assert set(over) <= set(a), over
    a.update(over)
    return fn(*a.values())


DROP = dict(y=A, ld_y=64, r=A + STEP, ld_r=64, p=0.1, seed=A + 2 * STEP, T=4, H=64, dtype=0, out=A + 3 * STEP, ld_out=64,
            stream=None)


@pytest.mark.parametrize("over,code", [
    (dict(dtype=3), -10), (dict(p=-0.1), -10), (dict(p=1.5), -10), (dict(p=math.nan), -10), (dict(T=-1), -2),
    (dict(T=2 ** 31), -2), (dict(H=0), -2), (dict(H=60), -2), (dict(ld_y=56), -2), (dict(ld_y=68), -2), (dict(ld_r=32), -2),
    (dict(ld_out=65), -2), (dict(y=None), -1), (dict(out=None), -1), (dict(seed=None), -1), (dict(y=A + 8), -3),
    (dict(r=A + STEP + 4), -3), (dict(seed=A + 4), -3), (dict(out=A, ld_out=72), -9), (dict(out=A + STEP + 16), -9),
    (dict(out=A + 2 * STEP - 16), -9), (dict(T=0, y=None, out=None), 0)])
def test_dropout_refusals(L, over, code):
    assert _call(L.mhc_dropout, DROP, over) == code


def test_binding_refuses_host_tensors_and_types():
    f = torch.zeros
    with pytest.raises(B.MhcError) as e:
        B.mhc_dropout(f(4, 64), f(4, 64), f(2), stream=0)
    assert e.value.code in (-2, -10)
    with pytest.raises(B.MhcError) as e:
        B.mhc_dropout(f(4, 64), f(4, 64), f(2, dtype=torch.int64), stream=0)
    assert e.value.code == -10 and "GPU" in str(e.value)


# ---------------------------------------- the test implementations themselves --
def test_philox_known_answers():
    # the generator's published test vectors (zeros, ones, digits of pi)
    assert R.philox((0, 0, 0, 0), (0, 0)) == (0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8)
    f = 0xFFFFFFFF
    assert R.philox((f, f, f, f), (f, f)) == (0x408F276D, 0x41C83B0E, 0xA20BC7C6, 0x6D5451FD)
    assert R.philox((0x243F6A88, 0x85A308D3, 0x13198A2E, 0x03707344), (0xA4093822, 0x299F31D0)) == \
        (0xD16CFE09, 0x94FDCCEB, 0x5001E420, 0x24126EA1)


def test_dropout_reference_by_hand():
    y, r = torch.ones(2, 8), torch.full((2, 8), 3.0)
    assert torch.equal(R.dropout(y, r, 0.0, 1, 2)[0], torch.full((2, 8), 4.0).double())
    assert torch.equal(R.dropout(y, None, 1.0, 1, 2)[0], torch.zeros(2, 8).double())
    out = R.dropout(torch.ones(100, 40), None, 0.25, 7, 9)[0]
    assert set(out.unique().tolist()) == {0.0, 4 / 3} and abs(float((out == 0).double().mean()) - 0.25) < 5 * (0.1875 / 4000) ** 0.5


GLU = dict(x=A, ld_x=64, w=A + STEP, add=A + 2 * STEP, ld_add=256, act=0, T=4, H=64, F=128, dtype=0, gu=A + 3 * STEP,
           h=A + 4 * STEP, ld_h=128, ws=A + 5 * STEP, ws_bytes=1 << 27, stream=None)


@pytest.mark.parametrize("over,code", [
    (dict(dtype=2), -10), (dict(dtype=5), -10), (dict(act=4), -10), (dict(act=-1), -10), (dict(T=-1), -2), (dict(T=2 ** 31), -2),
    (dict(H=60), -2), (dict(H=0), -2), (dict(F=132, ld_h=136), -2), (dict(F=0), -2), (dict(F=2 ** 21, ld_h=2 ** 21, ld_add=2 ** 22), -2),
    (dict(ld_x=56), -2), (dict(ld_x=68), -2), (dict(ld_add=128), -2), (dict(ld_add=260), -2), (dict(ld_h=120), -2),
    (dict(x=None), -1), (dict(w=None), -1), (dict(h=None), -1), (dict(x=A + 8), -3), (dict(w=A + STEP + 2), -3),
    (dict(add=A + 2 * STEP + 4), -3), (dict(gu=A + 3 * STEP + 8), -3), (dict(h=A + 4 * STEP + 8), -3), (dict(ws=A + 5 * STEP + 4), -3),
    (dict(ws=None), -5), (dict(ws_bytes=100), -5), (dict(h=A), -9), (dict(h=A + STEP), -9), (dict(gu=A + 2 * STEP), -9),
    (dict(gu=A + 4 * STEP), -9), (dict(ws=A + 4 * STEP), -9), (dict(ws=A), -9), (dict(T=0, x=None, h=None, ws=None), 0)])
def test_glu_refusals(L, over, code):
    assert _call(L.mhc_glu, GLU, over) == code


def test_glu_reference_is_torch():
    g = torch.Generator().manual_seed(4)
    x, w = torch.randn(3, 8, generator=g).double(), torch.randn(10, 8, generator=g).double()
    f = torch.nn.functional
    for name, fn in (("silu", f.silu), ("gelu", f.gelu), ("gelu_tanh", lambda v: f.gelu(v, approximate="tanh")), ("relu", f.relu)):
        a, b = (x @ w.t())[:, :5].requires_grad_(), (x @ w.t())[:, 5:]
        assert torch.allclose(R.glu(x, w, None, name)[0]["h"], (fn(a) * b).detach(), rtol=1e-9, atol=1e-12)
        assert torch.allclose(R.act(a.detach(), name)[1], torch.autograd.grad(fn(a).sum(), a)[0], rtol=1e-9, atol=1e-12)


GGRAD = dict(dh=A, gu=A + STEP, x=A + 2 * STEP, ld_x=64, w=A + 3 * STEP, act=0, T=4, H=64, F=128, dtype=0, dgu=A + 4 * STEP,
             dx=A + 5 * STEP, dw=A + 6 * STEP, dw_dtype=2, acc=0, ws=A + 7 * STEP, ws_bytes=1 << 27, stream=None)


@pytest.mark.parametrize("over,code", [
    (dict(dtype=2), -10), (dict(dw_dtype=1), -10), (dict(act=9), -10), (dict(T=-1), -2), (dict(H=12), -2), (dict(F=4), -2),
    (dict(ld_x=60), -2), (dict(ld_x=32), -2), (dict(dh=None), -1), (dict(gu=None), -1), (dict(dgu=None), -1), (dict(x=None), -1),
    (dict(w=None), -1), (dict(dh=A + 8), -3), (dict(dw=A + 6 * STEP + 4), -3), (dict(ws=A + 7 * STEP + 2), -3), (dict(ws=None), -5),
    (dict(ws_bytes=10), -5), (dict(dgu=A + STEP), -9), (dict(dx=A + 2 * STEP), -9), (dict(dw=A + 3 * STEP), -9), (dict(dx=A + 4 * STEP), -9),
    (dict(dw=A + 5 * STEP), -9), (dict(ws=A), -9), (dict(ws=A + 4 * STEP), -9), (dict(T=0, acc=1, dh=None, dgu=None, ws=None), 0),
    (dict(T=0, dw=None, dh=None, dgu=None, ws=None), 0)])
def test_glu_grad_refusals(L, over, code):
    assert _call(L.mhc_glu_grad, GGRAD, over) == code


def test_glu_reference_gradient_is_the_derivative():
    g = torch.Generator().manual_seed(5)
    n = lambda *s: torch.randn(*s, generator=g, dtype=torch.float64)  # noqa: E731
    x, w, dh = n(4, 6).requires_grad_(), n(10, 6).requires_grad_(), n(4, 5)
    for name in R.ACTS:
        gu = x @ w.t()
        h = R.act(gu[:, :5], name)[0] * gu[:, 5:]
        want = torch.autograd.grad((h * dh).sum(), (gu, x, w))
        got = R.glu_grad(dh, gu.detach(), x.detach(), w.detach(), name, torch.bfloat16)[0]
        for k, v in zip(("dgu", "dx", "dw"), want):
            assert torch.allclose(got[k], v, rtol=1e-9, atol=1e-11), (name, k)


LORA = dict(x=A, ld_x=64, a=A + STEP, b=A + 2 * STEP, index=A + 3 * STEP, scale=A + 4 * STEP, T=4, H=64, N=128, R=16, n=3, dtype=0,
            base=A + 5 * STEP, ld_base=128, out=A + 6 * STEP, ld_out=128, ws=A + 7 * STEP, ws_bytes=1 << 24, stream=None)


@pytest.mark.parametrize("over,code", [
    (dict(dtype=2), -10), (dict(T=-1), -2), (dict(H=4), -2), (dict(N=12), -2), (dict(R=0), -2), (dict(R=12), -2), (dict(R=264), -2),
    (dict(n=-1), -2), (dict(ld_x=60), -2), (dict(ld_base=120), -2), (dict(ld_out=129), -2), (dict(x=None), -1), (dict(a=None), -1),
    (dict(b=None), -1), (dict(index=None), -1), (dict(out=None), -1), (dict(x=A + 8), -3), (dict(b=A + 2 * STEP + 4), -3),
    (dict(index=A + 3 * STEP + 2), -3), (dict(scale=A + 4 * STEP + 1), -3), (dict(ws=None), -5), (dict(ws_bytes=100), -5), (dict(n=2 ** 21), -2),
    (dict(out=A), -9), (dict(out=A + 2 * STEP), -9), (dict(out=A + 5 * STEP + 16), -9), (dict(out=A + 5 * STEP, ld_out=136), -9),
    (dict(ws=A + 5 * STEP), -9), (dict(ws=A + 6 * STEP), -9), (dict(ws=A + 3 * STEP), -9), (dict(T=0, x=None, out=None, ws=None), 0)])
def test_lora_refusals(L, over, code):
    assert _call(L.mhc_lora, LORA, over) == code


def test_lora_workspace_grows(L):
    sizes = [L.mhc_lora_workspace_bytes(t, 16) for t in (0, 1, 64, 2432, 2500, 40000, 10 ** 6)]
    assert sizes == sorted(sizes) and sizes[0] == 0 and sizes[-1] >= 10 ** 6 * 64


def test_lora_reference_by_hand():
    x = torch.tensor([[1.0, 2.0], [3.0, 4.0], [5.0, 6.0]])
    a, b = torch.tensor([[[1.0, 0.0]], [[0.0, 1.0]]]), torch.tensor([[[2.0], [0.0]], [[1.0], [1.0]]])
    out, _ = R.lora(x, a, b, torch.tensor([1, 0, -1]), torch.tensor([0.5, 10.0]), torch.ones(3, 2))
    assert out.tolist() == [[21.0, 21.0], [4.0, 1.0], [1.0, 1.0]]
