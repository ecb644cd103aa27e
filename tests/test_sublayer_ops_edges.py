"""The operators inside a block where they can go wrong: no adapters at all, one buffer as the workspace of all of
them, pre-activations whose squares leave fp32, and sums of whole numbers, which have one value in whatever order they
are added."""
import os
import sys

import pytest
import torch

from mhc_residual_seam_gb300 import binding as B

import sublayer_case as R
import sublayer_exact_case as X

pytestmark = pytest.mark.gpu

BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    B.lib()


def workspace(n):
    ws = torch.full((max(n, 16),), 0xA5, dtype=torch.uint8, device="cuda")
    B.mhc_workspace_init(ws)
    return ws


def full(*shape, dtype=BF16):
    return torch.full(shape, 7.0, dtype=dtype, device="cuda")


# --------------------------------------------------------- no adapters at all --
@pytest.mark.parametrize("rank", [16, 64, 256])
@pytest.mark.parametrize("T", [1, 64, 65, 1500])
def test_lora_without_adapters(T, rank):
    H, N = 136, 264
    x = torch.full((T, H), float("nan"), dtype=BF16, device="cuda")  # (nothing reads it)
    a, b = torch.empty(0, rank, H, dtype=BF16, device="cuda"), torch.empty(0, N, rank, dtype=BF16, device="cuda")
    index = (torch.arange(T) % 5 - 2).int().cuda()
    base = torch.randn(T, N, generator=torch.Generator().manual_seed(T)).to(BF16).cuda()
    ws = workspace(B.mhc_lora_workspace_bytes(T, rank))
    out = full(T, N)
    B.mhc_lora(x, a, b, index, out, ws, base=base)
    assert torch.equal(out, base)
    B.mhc_lora(x, a, b, index, out, ws)
    assert not bool(out.any())
    again = base.clone()
    B.mhc_lora(x, a, b, index, again, ws, scale=torch.empty(0, device="cuda"), base=again)
    assert torch.equal(again, base)
    B.mhc_check_status(ws)


# ------------------------------------------------- one buffer for all of them --
def test_one_buffer_for_projections_and_adapters():
    # the projections' counters outlive an adapter's call in the same buffer
    sizes = [(130, 8192, 264), (9, 5120, 2000), (1100, 2048, 5000)]  # tiles cut along H, in both forms
    lora = [(70, 16), (8192, 64), (20, 256), (3000, 8)]
    ws = workspace(max([B.mhc_glu_workspace_bytes(*s) for s in sizes] + [B.mhc_lora_workspace_bytes(*s) for s in lora]))
    g = torch.Generator(device="cuda").manual_seed(1)
    normal = lambda *s: torch.empty(*s, dtype=BF16, device="cuda").normal_(generator=g)  # noqa: E731
    jobs = []
    for T, H, F in sizes:
        x, w, add = X.glu_inputs(T, H, F, BF16, "cuda")
        jobs.append((x, w, add, X.glu(x, w, add, BF16)[0]))
    dh, gu, gx, gw = X.grad_inputs(700, 2920, 1000, BF16, "cuda")
    want = [t.to(BF16) for t in X.grad(dh, gu, gx, gw)]
    for T, rank in lora:
        lx, la, lb = normal(T, 264), normal(3, rank, 264), normal(3, 136, rank)
        index, out = (torch.arange(T, device="cuda") % 4 - 1).int(), full(T, 136)
        for x, w, add, h in jobs:
            B.mhc_lora(lx, la, lb, index, out, ws)
            got = full(*h.shape)
            B.mhc_glu(x, w, got, ws, add=add, act=B.MHC_ACT_RELU)
            assert torch.equal(got, h)
        B.mhc_lora(lx, la, lb, index, out, ws)
        got = [full(*t.shape) for t in want]
        B.mhc_glu_grad(dh, gu, gx, gw, *got, ws, act=B.MHC_ACT_RELU)
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    B.mhc_check_status(ws)


# ----------------------------------- pre-activations whose squares leave fp32 --
@pytest.mark.parametrize("act", range(4))
def test_gradient_of_huge_preactivations(act):
    g = torch.tensor([1e15, 1e19, 2e19, 1e25, 3e38, 1e5, 40.0, 1.0], dtype=BF16)
    g = torch.stack([g, -g])
    gu = torch.cat([g, torch.ones(2, 8, dtype=BF16)], 1)
    dh, x, w = torch.ones(2, 8, dtype=BF16), torch.ones(2, 8, dtype=BF16), torch.ones(16, 8, dtype=BF16)
    dgu = full(2, 16)
    B.mhc_glu_grad(dh.cuda(), gu.cuda(), None, None, dgu, None, None, workspace(B.mhc_glu_workspace_bytes(2, 8, 8)), act=act)
    name = R.ACTS[act]
    dgu = dgu.cpu().double()
    a, da, _ = R.act(g, name)  # (far out the activation is g or 0 and its derivative 1 or 0)
    for got, want in ((dgu[:, :8], da), (dgu[:, 8:], a)):
        # one rounding to bf16, and for g = 1 and -1 some fp32 ones of terms of about 1
        assert torch.allclose(got, want, rtol=2.0 ** -8, atol=2.0 ** -18)
    gu[:, 0] = float("nan")  # a NaN stays one
    B.mhc_glu_grad(dh.cuda(), gu.cuda(), None, None, out := full(2, 16), None, None,
                   workspace(B.mhc_glu_workspace_bytes(2, 8, 8)), act=act)
    assert bool(torch.isnan(out[:, 8]).all()) and (name == "relu" or bool(torch.isnan(out[:, 0]).all()))
    assert torch.equal(out.cpu().double()[:, 1:8], dgu[:, 1:8])


# ---------------------------------------------------- sums of whole numbers --
@pytest.mark.parametrize("T,H,F", X.GLU)
@pytest.mark.parametrize("dtype", [BF16, F16])
def test_glu_of_whole_numbers(T, H, F, dtype):
    x, w, add = X.glu_inputs(T, H, F, dtype, "cuda")
    h, gu = X.glu(x, w, add, dtype)
    ws = workspace(B.mhc_glu_workspace_bytes(T, H, F))
    for keep in (True, False):
        got, kept = full(T, F, dtype=dtype), full(T, 2 * F, dtype=dtype) if keep else None
        B.mhc_glu(x, w, got, ws, add=add, gu=kept, act=B.MHC_ACT_RELU)
        assert torch.equal(got, h) and (not keep or torch.equal(kept, gu))
    B.mhc_check_status(ws)


@pytest.mark.parametrize("T,H,F", X.GRAD)
@pytest.mark.parametrize("dtype", [BF16, F16])
def test_glu_grad_of_whole_numbers(T, H, F, dtype):
    dh, gu, x, w = X.grad_inputs(T, H, F, dtype, "cuda")
    dgu, dx, dw = X.grad(dh, gu, x, w)
    ws = workspace(B.mhc_glu_workspace_bytes(T, H, F))
    old = X.whole(torch.Generator().manual_seed(1), 2 * F, H, most=100).cuda()
    for wdt in (dtype, F32):
        for add in (False, True):
            to = old.to(wdt, copy=True)
            want = (dw + old.double() if add else dw).to(wdt)
            got = [full(T, 2 * F, dtype=dtype), full(T, H, dtype=dtype)]
            B.mhc_glu_grad(dh, gu, x, w, *got, to, ws, act=B.MHC_ACT_RELU, accumulate=add)
            assert torch.equal(got[0], dgu.to(dtype)) and torch.equal(got[1], dx.to(dtype)) and torch.equal(to, want)
            # each product by itself: its tiles are cut at other places
            to = old.to(wdt, copy=True)
            B.mhc_glu_grad(dh, gu, x, None, got[0], None, to, ws, act=B.MHC_ACT_RELU, accumulate=add)
            assert torch.equal(to, want)
    alone = full(T, H, dtype=dtype)
    B.mhc_glu_grad(dh, gu, None, w, got[0], alone, None, ws, act=B.MHC_ACT_RELU)
    assert torch.equal(alone, dx.to(dtype))
    B.mhc_check_status(ws)


@pytest.mark.parametrize("T,H,N,rank,n", X.LORA)
@pytest.mark.parametrize("dtype", [BF16, F16])
def test_lora_of_whole_numbers(T, H, N, rank, n, dtype):
    x, a, b, index, scale, base = X.lora_inputs(T, H, N, rank, n, dtype, "cuda")
    ws = workspace(B.mhc_lora_workspace_bytes(T, rank))
    out = full(T, N, dtype=dtype)
    B.mhc_lora(x, a, b, index, out, ws, scale=scale, base=base)
    assert torch.equal(out, X.lora(x, a, b, index, scale, base).to(dtype))
    B.mhc_lora(x, a, b, index, out, ws)
    assert torch.equal(out, X.lora(x, a, b, index, torch.ones_like(scale), torch.zeros_like(base)).to(dtype))
    B.mhc_check_status(ws)


# ---------------------------------------------------------- the smoke test --
def test_smoke_initialises_every_workspace(monkeypatch):
    sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
    import __graft_entry__ as entry
    ready = set()
    init = B.mhc_workspace_init
    monkeypatch.setattr(B, "mhc_workspace_init", lambda ws, *a: (init(ws, *a), ready.add((ws.data_ptr(), ws.numel()))))
    for name, at in (("mhc_lora", 5), ("mhc_glu", 3), ("mhc_glu_grad", 7)):
        def call(*a, f=getattr(B, name), at=at, **k):
            assert (a[at].data_ptr(), a[at].numel()) in ready, f
            f(*a, **k)
        monkeypatch.setattr(B, name, call)
    entry._smoke_sublayer(torch, B)
