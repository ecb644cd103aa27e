"""Refusals of the operators around the seam, and checks of their 64-bit test
implementations, without a GPU.  The addresses below are fake; every call
fails its checks before anything touches them."""
import math

import pytest
import torch

from mhc_residual_seam_gb300 import binding as B

import block_case as R

A = 0x10000000  # 256-byte aligned, never dereferenced
STEP = 0x1000000


@pytest.fixture(scope="module")
def L():
    return B.lib()


def _call(fn, order, base, over):
    a = dict(base)
    assert set(over) <= set(a), over
    a.update(over)
    return fn(*[a[k] for k in order])


EMBED = dict(ids=A, id_bytes=8, table=A + STEP, table_ld=64, V=100, first=0, scale=1.0, T=4, H=64, streams=4, dtype=0,
             out=A + 2 * STEP, stream=None)


@pytest.mark.parametrize("over,code", [
    (dict(dtype=3), -10), (dict(id_bytes=2), -10), (dict(T=-1), -2), (dict(H=60), -2), (dict(H=0), -2), (dict(V=-1), -2),
    (dict(streams=0), -2), (dict(streams=65), -2), (dict(table_ld=56), -2), (dict(table_ld=68), -2), (dict(ids=None), -1),
    (dict(table=None), -1), (dict(out=None), -1), (dict(out=A + 2 * STEP + 8), -3), (dict(table=A + 4), -3),
    (dict(ids=A + 4), -3), (dict(out=A + STEP), -9), (dict(out=A), -9), (dict(T=0, ids=None, out=None), 0)])
def test_embed_refusals(L, over, code):
    assert _call(L.mhc_embed, EMBED, EMBED, over) == code


GRAD = dict(ids=A, id_bytes=8, dout=A + STEP, dtype=0, scale=1.0, T=4, H=64, streams=4, V=100, first=0, pad=None, acc=0,
            dtable=A + 2 * STEP, grad=2, ld=64, ws=A + 3 * STEP, ws_bytes=1 << 24, stream=None)


@pytest.mark.parametrize("over,code", [
    (dict(dtype=5), -10), (dict(grad=1), -10), (dict(grad=-1), -10), (dict(id_bytes=1), -10), (dict(T=-1), -2),
    (dict(T=2 ** 31), -2), (dict(V=2 ** 31), -2), (dict(H=4), -2), (dict(streams=0), -2), (dict(ld=60), -2), (dict(ld=32), -2),
    (dict(ids=None), -1), (dict(dout=None), -1), (dict(dtable=None), -1), (dict(dout=A + STEP + 2), -3), (dict(ws=A + 8), -3),
    (dict(ws=None), -5), (dict(ws_bytes=255), -5), (dict(dtable=A + STEP), -9), (dict(ws=A + 2 * STEP), -9),
    (dict(ws=A), -9), (dict(V=0, ids=None), 0), (dict(T=0, acc=1, ids=None, dout=None, ws=None), 0)])
def test_embed_grad_refusals(L, over, code):
    assert _call(L.mhc_embed_grad, GRAD, GRAD, over) == code


NORM = dict(y=A, ld_y=64, r=A + STEP, ld_r=64, gpost=A + 2 * STEP, gate=A + 3 * STEP, mode=1, gpre=A + 4 * STEP, scale=1.0,
            eps=1e-6, T=4, H=64, dtype=0, ro=A + 5 * STEP, ld_ro=64, norm=A + 6 * STEP, ld_n=64, rp=A + 7 * STEP,
            rq=A + 8 * STEP, stream=None)


@pytest.mark.parametrize("over,code", [
    (dict(dtype=9), -10), (dict(mode=3), -10), (dict(mode=-1), -10), (dict(eps=-1.0), -10), (dict(eps=math.nan), -10),
    (dict(T=-1), -2), (dict(H=12), -2), (dict(H=16392), -2), (dict(ld_y=60), -2), (dict(ld_r=56), -2), (dict(ld_n=0), -2),
    (dict(r=None, y=None, gpost=None, gate=None, mode=0), -1), (dict(ro=None), -1), (dict(norm=None), -1), (dict(rp=None), -1), (dict(rq=None), -1),
    (dict(gate=None), -1), (dict(mode=0), -1), (dict(y=None), -4), (dict(y=None, gpost=None, gate=None, mode=0, gpre=None), -4),
    (dict(y=A + 8), -3), (dict(gpre=A + 4 * STEP + 2), -3), (dict(rp=A + 7 * STEP + 2), -3), (dict(ro=A), -9),
    (dict(ro=A + STEP, ld_ro=72), -9), (dict(ro=A + STEP + 16), -9), (dict(norm=A + 5 * STEP), -9), (dict(norm=A + STEP), -9),
    (dict(rq=A + 7 * STEP), -9), (dict(gate=A + 5 * STEP), -9), (dict(T=0, r=None, ro=None), 0)])
def test_block_norm_refusals(L, over, code):
    assert _call(L.mhc_block_norm, NORM, NORM, over) == code


BGRAD = dict(dro=A, dn=A + STEP, y=A + 2 * STEP, ro=A + 3 * STEP, gpost=A + 4 * STEP, gate=A + 5 * STEP, mode=2,
             gpre=A + 6 * STEP, rp=A + 7 * STEP, rq=A + 8 * STEP, scale=1.0, T=4, H=64, dtype=0, dy=A + 9 * STEP,
             dr=A + 10 * STEP, dgp=A + 11 * STEP, dgt=A + 12 * STEP, dgq=A + 13 * STEP, ws=A + 14 * STEP, ws_bytes=1 << 24,
             stream=None)


@pytest.mark.parametrize("over,code", [
    (dict(dtype=3), -10), (dict(mode=7), -10), (dict(T=-2), -2), (dict(H=20), -2), (dict(dn=None), -1), (dict(ro=None), -1),
    (dict(rq=None), -1), (dict(rp=None), -1), (dict(dr=None, y=None), -1), (dict(dy=None), -1), (dict(dgp=None), -1),
    (dict(dgt=None), -1), (dict(dgq=None), -1), (dict(gate=None), -1), (dict(mode=0), -1), (dict(dro=None, gpre=None), -1),
    (dict(y=None), -4), (dict(dy=A + 9 * STEP + 2), -3), (dict(dgp=A + 2), -3), (dict(ws=A + 8), -3), (dict(ws=None), -5),
    (dict(ws_bytes=100), -5), (dict(dy=A), -9), (dict(dr=A + 9 * STEP), -9), (dict(ws=A + 2 * STEP), -9), (dict(dgp=A + 13 * STEP), -9)])
def test_block_norm_grad_refusals(L, over, code):
    assert _call(L.mhc_block_norm_grad, BGRAD, BGRAD, over) == code


ROUTE = dict(logits=A, ld=64, dtype=2, bias=None, score=1, E=64, groups=8, top=4, k=8, renorm=1, scale=1.0, T=4,
             idx=A + STEP, w=A + 2 * STEP, counts=A + 3 * STEP, ws=A + 4 * STEP, ws_bytes=4096, stream=None)


@pytest.mark.parametrize("over,code", [
    (dict(dtype=4), -10), (dict(score=2), -10), (dict(scale=math.nan), -10), (dict(T=-1), -2), (dict(E=0), -2),
    (dict(E=1032, ld=1032), -2), (dict(k=0), -2), (dict(k=33), -2), (dict(E=4, ld=64, groups=1, top=1, k=5), -2),
    (dict(ld=63), -2), (dict(groups=0), -2), (dict(groups=7), -2), (dict(groups=64, top=9), -2), (dict(top=9), -2),
    (dict(top=0), -2), (dict(top=1, k=9), -2), (dict(logits=None), -1), (dict(idx=None), -1), (dict(w=None), -1),
    (dict(logits=A + 2), -3), (dict(idx=A + STEP + 1), -3), (dict(counts=A + 3 * STEP + 1), -3), (dict(ws=None), -5),
    (dict(ws_bytes=100), -5), (dict(idx=A), -9), (dict(w=A + STEP), -9), (dict(ws=A + 3 * STEP), -9), (dict(bias=A + 2 * STEP), -9),
    (dict(T=0, counts=None, ws=None, logits=None), 0)])
def test_route_refusals(L, over, code):
    assert _call(L.mhc_route, ROUTE, ROUTE, over) == code


RGRAD = dict(dw=A, logits=A + STEP, ld=64, dtype=2, idx=A + 2 * STEP, score=1, E=64, k=8, renorm=1, scale=1.0, T=4,
             dl=A + 3 * STEP, ld_d=64, stream=None)


@pytest.mark.parametrize("over,code", [
    (dict(dtype=4), -10), (dict(score=-1), -10), (dict(E=2000, ld=2000, ld_d=2000), -2), (dict(k=40), -2), (dict(ld_d=63), -2),
    (dict(dw=None), -1), (dict(logits=None), -1), (dict(idx=None), -1), (dict(dl=None), -1), (dict(dl=A + 3 * STEP + 2), -3),
    (dict(dl=A + STEP), -9), (dict(dl=A), -9), (dict(dl=A + 2 * STEP), -9), (dict(T=0, dw=None), 0)])
def test_route_grad_refusals(L, over, code):
    assert _call(L.mhc_route_grad, RGRAD, RGRAD, over) == code


def test_binding_refuses_host_tensors_types_and_shapes():
    f = torch.zeros
    with pytest.raises(B.MhcError) as e:
        B.mhc_embed(f(4, dtype=torch.int64), f(10, 64), f(4, 64))
    assert e.value.code == -10 and "GPU" in str(e.value)
    with pytest.raises(B.MhcError):
        B.mhc_route(f(4, 8), None, f(4, 2, dtype=torch.int32), f(4, 2), stream=0)
    with pytest.raises(B.MhcError):
        B.mhc_block_norm(None, f(4, 64), None, None, f(64), None, f(4, 64), None, f(4), stream=0)


def test_workspace_sizes_follow_the_plan(L):
    # sorted keys and tokens twice (256-byte steps), counts, bounds and one carry row per chunk
    assert L.mhc_embed_grad_workspace_bytes(0, 10, 64) == 256
    a, b = L.mhc_embed_grad_workspace_bytes(1000, 1000, 64), L.mhc_embed_grad_workspace_bytes(100000, 1000, 64)
    assert 256 + 4 * 4096 < a < b and b > 16 * 100000
    assert L.mhc_block_norm_grad_workspace_bytes(0, 64) == 0
    # two fp32 rows of column sums per CTA: one CTA for a few rows, all that are resident for many
    assert L.mhc_block_norm_grad_workspace_bytes(5, 64) == 2 * 64 * 4
    assert L.mhc_block_norm_grad_workspace_bytes(10 ** 6, 5120) <= 304 * 2 * 5120 * 4
    assert L.mhc_block_norm_grad_workspace_bytes(10 ** 6, 16384) <= 152 * 2 * 16384 * 4
    assert L.mhc_route_workspace_bytes(256) == 256 + 1024


# ---------------------------------------- the test implementations themselves --
def test_block_norm_reference_gradient_is_the_derivative():
    g = torch.Generator().manual_seed(1)
    n = lambda *s: torch.randn(*s, generator=g, dtype=torch.float64)  # noqa: E731
    for mode in ("none", "channel", "token"):
        for post in (False, True):
            T, H = 3, 16
            v = {"y": n(T, H), "r": n(T, H), "gp": 1 + 0.1 * n(H) if post else None, "gq": 1 + 0.1 * n(H),
                 "gate": {"none": None, "channel": n(H), "token": n(T)}[mode]}
            leaf = {k: None if x is None else x.clone().requires_grad_() for k, x in v.items()}
            f = R.block_norm(leaf["y"], leaf["r"], leaf["gp"], leaf["gate"], mode, leaf["gq"], 0.5, 1e-6)
            do, dn = n(T, H), n(T, H)
            ((f["r_out"] * do).sum() + (f["norm"] * dn).sum()).backward()
            f = {k: x.detach() for k, x in f.items()}
            ref = R.block_norm_grad(do, dn, v["y"], f["r_out"], v["gp"], v["gate"], mode, v["gq"], f.get("rstd_post"),
                                    f["rstd_pre"], 0.5)
            for k, name in (("y", "dy"), ("r", "dr"), ("gp", "dgamma_post"), ("gq", "dgamma_pre"), ("gate", "dgate")):
                if leaf[k] is not None:
                    assert torch.allclose(leaf[k].grad, ref[name], rtol=1e-10, atol=1e-12), (mode, post, k)


def test_route_reference_gradient_is_the_derivative():
    g = torch.Generator().manual_seed(2)
    l = torch.randn(5, 9, generator=g, dtype=torch.float64)
    idx = torch.stack([torch.randperm(9, generator=g)[:3] for _ in range(5)])
    dw = torch.randn(5, 3, generator=g, dtype=torch.float64)
    for sigmoid in (True, False):
        for renorm in (True, False):
            x = l.clone().requires_grad_()
            p = (torch.sigmoid(x) if sigmoid else torch.softmax(x, 1)).gather(1, idx)
            ((p / p.sum(1, keepdim=True) if renorm else p) * 1.5 * dw).sum().backward()
            assert torch.allclose(x.grad, R.route_grad(dw, l, idx, sigmoid, renorm, 1.5)[0], rtol=1e-10, atol=1e-12)


def test_route_reference_by_hand():
    l = torch.log(torch.tensor([[1.0, 2.0, 3.0, 4.0], [1.0, 1.0, 1.0, 1.0]]))
    idx, w, c, _ = R.route(l, None, False, 1, 1, 2, False, 1.0)
    assert idx.tolist() == [[3, 2], [0, 1]] and torch.allclose(w, torch.tensor([[0.4, 0.3], [0.25, 0.25]]).double())
    assert c.tolist() == [1, 1, 1, 1]
    idx, w, _, _ = R.route(l, torch.tensor([9.0, 0, 0, 0]), False, 2, 1, 2, True, 2.0)
    assert idx.tolist() == [[0, 1], [0, 1]] and torch.allclose(w[0], torch.tensor([2 / 3, 4 / 3]).double())
