"""The operators around the seam on the GPU (embedding, block norms, routing and
their gradients) against plain 64-bit implementations, with the bounds that
block_case.py derives."""
import math
import os
import subprocess
import sys

import pytest
import torch

from mhc_residual_seam_gb300 import binding as B

import block_case as R

pytestmark = pytest.mark.gpu

BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32
MODES = {"none": B.MHC_GATE_NONE, "channel": B.MHC_GATE_CHANNEL, "token": B.MHC_GATE_TOKEN}


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    B.lib()


def gen(seed):
    return torch.Generator().manual_seed(seed)


def normal(g, *shape, std=1.0, dtype=F32):
    return (std * torch.randn(*shape, generator=g)).to(dtype)


def dev(t):
    return None if t is None else t.cuda()


def workspace(n):
    # not zero: the workspaces without initialisation may hold anything
    return torch.full((max(n, 16),), 0xA5, dtype=torch.uint8, device="cuda")


# --------------------------------------------------------------- embedding --
@pytest.mark.parametrize("T,V,H,S,dtype,ids", [
    (1, 1, 8, 1, BF16, torch.int64), (7, 50, 40, 4, F16, torch.int32), (33, 1000, 136, 3, F32, torch.int64),
    (257, 513, 1032, 4, BF16, torch.int32), (64, 2000, 5120, 4, BF16, torch.int64)])
def test_embed(T, V, H, S, dtype, ids):
    g = gen(T + V)
    table = normal(g, V, H, dtype=dtype)
    i = torch.randint(0, V, (T,), generator=g).to(ids)
    out = torch.empty(T, S, H, dtype=dtype, device="cuda")
    B.mhc_embed(dev(i), dev(table), out, scale=1.75)
    # one fp32 product and one rounding: the same as torch's
    assert torch.equal(out.cpu(), (table.float() * 1.75).to(dtype)[i.long()][:, None].expand(T, S, H))
    R.check(out, R.embed(i, table, 1.75, 0, S), torch.zeros(T, S, H), what="embed")


def test_embed_outside_the_table_is_zero():
    V, H = 10, 64
    table = normal(gen(1), V, H, dtype=BF16).cuda()
    for dt, ids in ((torch.int64, [-2 ** 63, -100, 99, 100, 109, 110, 2 ** 40, 2 ** 63 - 1]),
                    (torch.int32, [-2 ** 31, -1, 99, 100, 109, 110, 2 ** 31 - 1])):
        i = torch.tensor(ids, dtype=dt)
        out = torch.full((len(ids), H), 7.0, dtype=BF16, device="cuda")
        B.mhc_embed(i.cuda(), table, out, first_id=100)
        for t, v in enumerate(ids):
            want = table[v - 100] if 100 <= v < 110 else torch.zeros(H, dtype=BF16, device="cuda")
            assert torch.equal(out[t], want), v


def test_embed_strided_table_and_no_tokens():
    big = normal(gen(2), 30, 128, dtype=F16).cuda()
    i = torch.tensor([3, 0, 29], device="cuda")
    out = torch.empty(3, 2, 64, dtype=F16, device="cuda")
    B.mhc_embed(i, big[:, 64:], out)
    assert torch.equal(out, big[i][:, None, 64:].expand(3, 2, 64))
    B.mhc_embed(i[:0], big, torch.empty(0, 128, dtype=F16, device="cuda"))


def _ids(g, T, V, kind):
    if kind == "skewed":
        return (torch.rand(T, generator=g).double().mul(math.log(V + 1)).exp().long() - 1).clamp_(0, V - 1)
    if kind == "one":
        return torch.full((T,), V - 1)
    return torch.randint(0, V, (T,), generator=g)


@pytest.mark.parametrize("T,V,H,S,dtype,grad,kind", [
    (1, 1, 8, 1, BF16, BF16, "any"), (5, 3, 40, 2, F16, F32, "any"), (100, 511, 64, 1, F32, F32, "any"),
    (100, 512, 64, 4, BF16, F32, "skewed"), (2047, 300, 72, 1, BF16, BF16, "skewed"),
    (2048, 40000, 8, 1, F16, F16, "any"), (2049, 7, 1032, 1, BF16, F32, "any"), (6000, 5000, 16, 2, F32, F32, "skewed"),
    (6001, 300000, 8, 1, BF16, F32, "skewed"), (4100, 1000, 24, 1, BF16, F32, "one"), (700, 900, 2056, 3, BF16, F32, "skewed"),
    (9000, 2, 40, 1, F32, F32, "any")])
def test_embed_grad(T, V, H, S, dtype, grad, kind):
    g = gen(T * 7 + V)
    i = _ids(g, T, V, kind)
    dout = normal(g, T, S, H, dtype=dtype)
    ref, terms, n = R.embed_grad(i, dout, V, 0.75)
    ws = workspace(B.mhc_embed_grad_workspace_bytes(T, V, H))
    out = torch.full((V, H), 3.0, dtype=grad, device="cuda")
    B.mhc_embed_grad(dev(i), dev(dout), out, ws, scale=0.75)
    R.check(out, ref, terms, n=n + 4, what="embed_grad")
    again = torch.full((V, H), 5.0, dtype=grad, device="cuda")
    B.mhc_embed_grad(dev(i.int()), dev(dout), again, ws, scale=0.75)
    assert torch.equal(out, again)  # the same bits whatever the timing and the ids' type


@pytest.mark.parametrize("T,V,kind", [(65536, 700, "skewed"), (65537, 100000, "skewed"), (300001, 3, "any"), (400000, 600000, "any")])
def test_embed_grad_of_many_tokens(T, V, kind):
    # small whole numbers: every order of the sum gives the same bits
    g = torch.Generator(device="cuda").manual_seed(T)
    i = _ids(gen(T), T, V, kind).cuda()
    dout = torch.randint(-2, 3, (T, 8), generator=g, device="cuda").float()
    out = torch.full((V, 8), 3.0, device="cuda")
    B.mhc_embed_grad(i, dout, out, workspace(B.mhc_embed_grad_workspace_bytes(T, V, 8)))
    assert torch.equal(out, torch.zeros(V, 8, device="cuda").index_add_(0, i, dout))


def test_embed_grad_shard_padding_accumulate():
    T, V, H, first = 3000, 100, 136, 250
    g = gen(5)
    i = torch.randint(-5, 600, (T,), generator=g)
    dout = normal(g, T, 2, H, dtype=BF16)
    old = normal(g, V, H)
    ref, terms, n = R.embed_grad(i, dout, V, 2.0, first=first, padding=260)
    ws = workspace(B.mhc_embed_grad_workspace_bytes(T, V, H))
    out = torch.empty(V, H, device="cuda")
    B.mhc_embed_grad(dev(i), dev(dout), out, ws, scale=2.0, first_id=first, padding_id=260)
    R.check(out, ref, terms, n=n + 4)
    assert not bool(out[10].any())
    add = old.cuda()
    i[(i >= first) & (i < first + 30)] = -1  # rows without tokens keep their value
    ref, terms, n = R.embed_grad(i, dout, V, 2.0, first=first, padding=300)
    B.mhc_embed_grad(dev(i), dev(dout), add, ws, scale=2.0, first_id=first, padding_id=300, accumulate=True)
    R.check(add, old.double() + ref, terms + old.abs(), n=n + 5)
    assert torch.equal(add[:30].cpu(), old[:30]) and torch.equal(add[50].cpu(), old[50])


def test_embed_grad_strided_no_tokens_and_none_valid():
    V, H = 37, 64
    big = torch.full((V, 2 * H), 9.0, device="cuda")
    ws = workspace(B.mhc_embed_grad_workspace_bytes(8, V, H))
    none = torch.empty(0, dtype=torch.int64, device="cuda")
    B.mhc_embed_grad(none, torch.empty(0, H, device="cuda"), big[:, :H], ws, accumulate=True)
    assert bool((big == 9).all())
    B.mhc_embed_grad(none, torch.empty(0, H, device="cuda"), big[:, :H], ws)
    assert not bool(big[:, :H].any()) and bool((big[:, H:] == 9).all())
    big.fill_(9.0)
    d = torch.ones(8, H, device="cuda")
    B.mhc_embed_grad(torch.full((8,), -100, device="cuda"), d, big[:, H:], ws)
    assert not bool(big[:, H:].any()) and bool((big[:, :H] == 9).all())


def test_embed_grad_against_differences():
    g = gen(6)
    T, V, H, S = 40, 9, 16, 2
    i = torch.randint(0, V, (T,), generator=g)
    up = normal(g, T, S, H)
    out = torch.empty(V, H, device="cuda")
    B.mhc_embed_grad(dev(i), dev(up), out, workspace(B.mhc_embed_grad_workspace_bytes(T, V, H)), scale=1.3)
    table = normal(g, V, H).double()
    for v, c in ((0, 0), (4, 7), (8, 15), (int(i[0]), 3)):
        lo, hi = table.clone(), table.clone()
        lo[v, c] -= 0.5
        hi[v, c] += 0.5  # linear: any step is exact
        d = ((R.embed(i, hi, 1.3, 0, S) - R.embed(i, lo, 1.3, 0, S)) * up.double()).sum()
        assert abs(float(out[v, c]) - float(d)) < 1e-4


# ------------------------------------------------------------- block norms --
def block_inputs(T, H, dtype, mode, post, pre, seed, y=True):
    g = gen(seed)
    d = {"y": normal(g, T, H, std=3, dtype=dtype) if y else None, "r": normal(g, T, H, std=2, dtype=dtype),
         "gamma_post": (1 + normal(g, H, std=0.1)).to(dtype) if post else None,
         "gamma_pre": (1 + normal(g, H, std=0.1)).to(dtype) if pre else None,
         "gate": {"none": None, "channel": (0.5 + normal(g, H, std=0.3)).to(dtype),
                  "token": 2 * torch.sigmoid(normal(g, T))}[mode],
         "dr_out": normal(g, T, H, dtype=dtype), "dnorm": normal(g, T, H, dtype=dtype) if pre else None}
    return d


def run_block(d, mode, scale=0.75, eps=1e-6, stream=None, inplace=False):
    T, H = d["r"].shape
    dt = d["r"].dtype
    e = lambda *s, t=F32: torch.full(s, 11.0, dtype=t, device="cuda")  # noqa: E731
    r = dev(d["r"])
    o = {"r_out": (r if inplace else e(T, H, t=dt)) if d["y"] is not None else None,
         "norm": e(T, H, t=dt) if d["gamma_pre"] is not None else None,
         "rstd_post": e(T) if d["gamma_post"] is not None else None,
         "rstd_pre": e(T) if d["gamma_pre"] is not None else None}
    B.mhc_block_norm(dev(d["y"]), r, dev(d["gamma_post"]), dev(d["gate"]), dev(d["gamma_pre"]), o["r_out"], o["norm"],
                     o["rstd_post"], o["rstd_pre"], gate_mode=MODES[mode], res_scale=scale, eps=eps, stream=stream)
    return o


def check_block(d, mode, o, scale=0.75, eps=1e-6):
    ref = R.block_norm(d["y"], d["r"], d["gamma_post"], d["gate"], mode, d["gamma_pre"], scale, eps)
    if o["r_out"] is not None:
        R.check(o["r_out"], ref["r_out"], ref["r_out_terms"], what="r_out")
    if o["rstd_post"] is not None:
        R.check(o["rstd_post"], ref["rstd_post"], ref["rstd_post"], what="rstd_post")
    if o["norm"] is not None:
        grow = ref["rho_grow"]
        R.check(o["norm"], ref["norm"], ref["norm_terms"] * grow[:, None], what="norm")
        R.check(o["rstd_pre"], ref["rstd_pre"], ref["rstd_pre"] * grow, what="rstd_pre")


FORMS = [(m, post, pre) for m in ("none", "channel", "token") for post in (False, True) for pre in (False, True)]


@pytest.mark.parametrize("mode,post,pre", FORMS)
@pytest.mark.parametrize("T,H,dtype", [(1, 8, BF16), (5, 264, F16), (6, 1000, F32), (3, 1032, BF16), (4, 5120, BF16)])
def test_block_norm_forms(T, H, dtype, mode, post, pre):
    d = block_inputs(T, H, dtype, mode, post, pre, T + H)
    check_block(d, mode, run_block(d, mode))


@pytest.mark.parametrize("H", [8, 64, 248, 256, 264, 512, 520, 1024, 2048, 4096, 4104, 7168, 8192, 8200, 16384])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_block_norm_widths(H, dtype):
    d = block_inputs(3, H, dtype, "channel", True, True, H)
    check_block(d, "channel", run_block(d, "channel"))


def test_block_norm_without_y_and_in_place():
    d = block_inputs(9, 640, BF16, "none", False, True, 3, y=False)
    check_block(d, "none", run_block(d, "none"))
    d = block_inputs(700, 1048, BF16, "token", True, True, 4)
    a, b = run_block(d, "token"), run_block(d, "token", inplace=True)
    for k in a:
        assert torch.equal(a[k], b[k]), k
    check_block(d, "token", b)


@pytest.mark.parametrize("T,H,dtype", [(5, 5120, BF16), (33, 264, F32), (9, 64, F16)])
def test_block_norm_without_residual(T, H, dtype):
    # r None: r_out = gate * p, which is what the seam takes as its Y; the gradient then has no dr
    for mode, post, pre in FORMS:
        d = block_inputs(T, H, dtype, mode, post, pre, 41)
        d["r"] = None
        e = lambda *s, t=F32: torch.full(s, 11.0, dtype=t, device="cuda")  # noqa: E731
        o = {"r_out": e(T, H, t=dtype), "norm": e(T, H, t=dtype) if pre else None, "rstd_post": e(T) if post else None,
             "rstd_pre": e(T) if pre else None}
        B.mhc_block_norm(dev(d["y"]), None, dev(d["gamma_post"]), dev(d["gate"]), dev(d["gamma_pre"]), o["r_out"], o["norm"],
                         o["rstd_post"], o["rstd_pre"], gate_mode=MODES[mode])
        check_block(d, mode, o, scale=1.0)
        d["r"] = d["y"]  # (the gradient's helpers take the shape from it)
        q = run_grad(d, mode, o)
        full = {k: v.clone() for k, v in q.items() if v is not None}
        dy, again = torch.empty_like(q["dy"]), {k: None if v is None else torch.empty_like(v) for k, v in q.items()}
        B.mhc_block_norm_grad(dev(d["dr_out"]), dev(d["dnorm"]), dev(d["y"]), o["r_out"], dev(d["gamma_post"]), dev(d["gate"]),
                              dev(d["gamma_pre"]), o["rstd_post"], o["rstd_pre"], dy, None, again["dgamma_post"],
                              again["dgate"], again["dgamma_pre"],
                              workspace(B.mhc_block_norm_grad_workspace_bytes(T, H)), gate_mode=MODES[mode], res_scale=0.75)
        R.check(dy, full["dy"].cpu().double(), full["dy"].cpu().double().abs(), n=8, what="dy")
        for k in ("dgamma_post", "dgate", "dgamma_pre"):
            if again[k] is not None:
                R.check(again[k], full[k].cpu().double(), full[k].cpu().double().abs(), n=8, what=k)


def test_block_norm_strided_streams():
    # r, r_out, y and norm as streams of [T,4,H] tensors: interleaved rows
    T, H = 21, 328
    g = gen(8)
    R4, O4 = normal(g, T, 4, H, dtype=BF16).cuda(), torch.zeros(T, 4, H, dtype=BF16, device="cuda")
    w = torch.ones(H, dtype=BF16, device="cuda")
    rp, rq = (torch.empty(T, device="cuda") for _ in range(2))
    before = R4.clone()
    B.mhc_block_norm(R4[:, 0], R4[:, 1], w, None, w, R4[:, 2], O4[:, 3], rp, rq)
    d = {"y": before[:, 0].cpu(), "r": before[:, 1].cpu(), "gamma_post": w.cpu(), "gamma_pre": w.cpu(), "gate": None}
    check_block(d, "none", {"r_out": R4[:, 2], "norm": O4[:, 3], "rstd_post": rp, "rstd_pre": rq}, scale=1.0)
    assert torch.equal(R4[:, [0, 1, 3]], before[:, [0, 1, 3]]) and not bool(O4[:, :3].any())
    with pytest.raises(B.MhcError) as e:  # half a row further on
        B.mhc_block_norm(R4[:, 0], R4[:, 1], w, None, w, R4.view(T, -1)[:, H // 2 - H // 2 % 8:][:, :H], O4[:, 3], rp, rq)
    assert e.value.code == -9


def test_block_norm_special_values():
    # a row of zeros stays zero, a row with NaN or inf stays that row's alone
    d = block_inputs(6, 1040, F32, "token", True, True, 9)
    d["y"][0] = 0
    d["r"][0] = 0
    d["y"][2, 5], d["r"][4, 7] = math.nan, math.inf
    o = run_block(d, "token")
    assert not bool(o["r_out"][0].any()) and not bool(o["norm"][0].any())
    assert math.isclose(float(o["rstd_pre"][0]), 1e3, rel_tol=1e-6)
    assert bool(torch.isnan(o["r_out"][2]).all()) and bool(torch.isnan(o["norm"][4, 7]))
    keep = [0, 1, 3, 5]
    check_block({k: v if v is None or k in ("gamma_post", "gamma_pre") else v[keep] for k, v in d.items()}, "token",
                {k: v[keep] for k, v in o.items()})


def run_grad(d, mode, o, scale=0.75, no_dr=False):
    T, H = d["r"].shape
    dt = d["r"].dtype
    e = lambda *s, t=F32: torch.full(s, 13.0, dtype=t, device="cuda")  # noqa: E731
    q = {"dy": e(T, H, t=dt) if d["y"] is not None else None, "dr": e(T, H, t=dt),
         "dgamma_post": e(H) if d["gamma_post"] is not None else None,
         "dgate": None if mode == "none" else e(T) if mode == "token" else e(H),
         "dgamma_pre": e(H) if d["gamma_pre"] is not None else None}
    x = dev(d["r"]) if d["y"] is None else o["r_out"]
    B.mhc_block_norm_grad(None if no_dr else dev(d["dr_out"]), dev(d["dnorm"]), dev(d["y"]), x, dev(d["gamma_post"]),
                          dev(d["gate"]), dev(d["gamma_pre"]), o["rstd_post"], o["rstd_pre"], q["dy"], q["dr"],
                          q["dgamma_post"], q["dgate"], q["dgamma_pre"],
                          workspace(B.mhc_block_norm_grad_workspace_bytes(T, H)), gate_mode=MODES[mode], res_scale=scale)
    return q


def check_grad(d, mode, o, q, scale=0.75, no_dr=False):
    cpu = lambda t: None if t is None else t.cpu()  # noqa: E731
    x = d["r"] if d["y"] is None else cpu(o["r_out"])
    ref = R.block_norm_grad(None if no_dr else d["dr_out"], d["dnorm"], d["y"], x, d["gamma_post"], d["gate"], mode,
                            d["gamma_pre"], cpu(o["rstd_post"]), cpu(o["rstd_pre"]), scale)
    T = d["r"].shape[0]
    for k, v in q.items():
        if v is not None:
            n = R.CHAIN + (T if v.dim() == 1 and k != "dgate" or mode == "channel" else d["r"].shape[1])
            R.check(v, ref[k], ref[k + "_terms"], n=n, what=k)


@pytest.mark.parametrize("mode,post,pre", FORMS)
@pytest.mark.parametrize("T,H,dtype", [(1, 8, BF16), (5, 264, F16), (307, 48, F32), (700, 1032, BF16), (2, 5120, BF16)])
def test_block_norm_grad_forms(T, H, dtype, mode, post, pre):
    d = block_inputs(T, H, dtype, mode, post, pre, T * 3 + H)
    o = run_block(d, mode)
    check_grad(d, mode, o, run_grad(d, mode, o))


@pytest.mark.parametrize("H", [64, 256, 264, 520, 1024, 2048, 4096, 4104, 8192, 8200, 16384])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_block_norm_grad_widths(H, dtype):
    d = block_inputs(5, H, dtype, "channel", True, True, H + 1)
    o = run_block(d, "channel")
    q = run_grad(d, "channel", o)
    check_grad(d, "channel", o, q)
    again = run_grad(d, "channel", o)
    assert all(torch.equal(q[k], again[k]) for k in q)


@pytest.mark.parametrize("T,H,dtype,mode", [(30011, 40, BF16, "token"), (20011, 264, F32, "channel"), (9001, 520, BF16, "channel"),
                                            (9001, 1024, BF16, "token"), (5003, 2056, F16, "channel")])
def test_block_norm_of_many_rows(T, H, dtype, mode):
    # more rows than the GPU has teams at a time
    d = block_inputs(T, H, dtype, mode, True, True, 51)
    o = run_block(d, mode)
    check_block(d, mode, o)
    check_grad(d, mode, o, run_grad(d, mode, o))


def test_block_norm_grad_without_y_dr_or_tokens():
    d = block_inputs(40, 640, BF16, "none", False, True, 21, y=False)
    o = run_block(d, "none")
    check_grad(d, "none", o, run_grad(d, "none", o, scale=1.0), scale=1.0)
    d = block_inputs(40, 2048, F32, "token", True, True, 22)
    o = run_block(d, "token")
    check_grad(d, "token", o, run_grad(d, "token", o, no_dr=True), no_dr=True)
    d = block_inputs(0, 64, F32, "channel", True, True, 23)
    q = run_grad(d, "channel", run_block(d, "channel"))
    assert not any(bool(q[k].any()) for k in ("dgamma_post", "dgamma_pre", "dgate"))


def test_block_norm_grad_against_differences():
    T, H, scale, eps, h = 3, 24, 0.75, 1e-6, 1e-4
    for mode, post, pre in FORMS:
        d = block_inputs(T, H, F32, mode, post, pre, 31)
        o = run_block(d, mode, scale, eps)
        q = run_grad(d, mode, o, scale)

        def loss(v):
            f = R.block_norm(v["y"], v["r"], v["gamma_post"], v["gate"], mode, v["gamma_pre"], scale, eps)
            return (f["r_out"] * d["dr_out"].double()).sum() + ((f["norm"] * d["dnorm"].double()).sum() if pre else 0)

        for name, got in (("y", "dy"), ("r", "dr"), ("gamma_post", "dgamma_post"), ("gamma_pre", "dgamma_pre"),
                          ("gate", "dgate")):
            if d[name] is None:
                continue
            flat = q[got].cpu().double().reshape(-1)
            for at in range(0, flat.numel(), max(1, flat.numel() // 5)):
                v = {k: None if x is None else x.double().clone() for k, x in d.items()}
                v[name].reshape(-1)[at] += h
                up = loss(v)
                v[name].reshape(-1)[at] -= 2 * h
                slope = (up - loss(v)) / (2 * h)
                # central differences are off by h^2 and 2^-52 / h, the kernel by fp32's roundings
                assert abs(float(slope) - float(flat[at])) < 2e-4 * (1 + abs(float(slope))), (mode, post, pre, name, at)


# ----------------------------------------------------------------- routing --
def run_route(l, bias, sigmoid, groups, top, k, renorm, scale=2.5, counts=True, ws=None, stream=None):
    T, E = l.shape
    idx = torch.full((T, k), -7, dtype=torch.int32, device="cuda")
    w = torch.full((T, k), 7.0, device="cuda")
    c = torch.full((E,), 7, dtype=torch.int32, device="cuda") if counts else None
    if counts and ws is None:
        ws = torch.empty(B.mhc_route_workspace_bytes(E), dtype=torch.uint8, device="cuda")
        B.mhc_workspace_init(ws)
    B.mhc_route(l if l.is_cuda else l.cuda(), dev(bias), idx, w, c, ws,
                score=B.MHC_SCORE_SIGMOID if sigmoid else B.MHC_SCORE_SOFTMAX, groups=groups, top_groups=top,
                renorm=renorm, scale=scale, stream=stream)
    return idx, w, c


def check_route(l, bias, sigmoid, groups, top, k, renorm, scale=2.5):
    idx, w, c = run_route(l, bias, sigmoid, groups, top, k, renorm, scale)
    ri, rw, rc, clear = R.route(l, bias, sigmoid, groups, top, k, renorm, scale)
    assert float(clear.double().mean()) > 0.9
    assert torch.equal(idx.cpu().long()[clear], ri[clear])
    # exp, a division and sums of at most 1024 terms (32 per lane, then 5 levels), all positive
    R.check(w[clear.cuda()], rw[clear], rw[clear], n=64, what="weights")
    got = idx.cpu().long()
    assert torch.equal(c.cpu().long(), torch.bincount(got[got >= 0], minlength=l.shape[1]))
    if bool(clear.all()):
        assert torch.equal(c.cpu().long(), rc)


@pytest.mark.parametrize("E,groups,top,k", [
    (1, 1, 1, 1), (8, 1, 1, 2), (8, 4, 2, 4), (60, 1, 1, 4), (64, 4, 1, 6), (64, 32, 3, 5), (160, 8, 3, 6), (256, 8, 4, 8),
    (256, 1, 1, 32), (384, 4, 3, 7), (512, 1, 1, 10), (1000, 10, 2, 9), (1024, 32, 8, 8), (33, 3, 2, 22), (20, 20, 5, 5)])
@pytest.mark.parametrize("sigmoid,renorm,bias", [(True, True, True), (False, False, False), (False, True, True)])
def test_route(E, groups, top, k, sigmoid, renorm, bias):
    g = gen(E + groups)
    l = normal(g, 45, E, std=1.5)
    l[7, torch.rand(E, generator=g) < 0.8] = -math.inf   # few experts left
    l[8] = -math.inf                                       # none left
    l[9, 0] = math.nan
    check_route(l, normal(g, E, std=0.1) if bias else None, sigmoid, groups, top, k, renorm)


@pytest.mark.parametrize("dtype", [BF16, F16])
def test_route_ties_go_to_the_lowest_index(dtype):
    g = gen(3)
    l = torch.randint(-3, 4, (70, 96), generator=g).to(dtype)  # many equal logits
    l[0] = 0
    l[1] = -0.0
    l[1, ::2] = 0.0
    for sigmoid in (True, False):
        check_route(l, None, sigmoid, 1, 1, 9, True)
        check_route(l, None, sigmoid, 6, 2, 9, True)


def test_route_infinities_and_rows_without_experts():
    l = torch.full((6, 40), -math.inf)
    l[1, 3] = math.inf
    l[2, [3, 9, 20]] = math.inf
    l[2, 5] = 1.0
    l[3] = math.nan
    l[4, 39] = -200.0  # its sigmoid is 0 in fp32
    l[5, :4] = torch.tensor([3e38, -3e38, 0.0, 1.0])
    for sigmoid, renorm in ((False, False), (False, True), (True, False), (True, True)):
        idx, w, c = run_route(l, None, sigmoid, 1, 1, 4, renorm, scale=1.0)
        ri, rw, rc, _ = R.route(l, None, sigmoid, 1, 1, 4, renorm, 1.0)
        if sigmoid and renorm:
            rw[4] = 0  # 0 / 0
        assert torch.equal(idx.cpu().long(), ri) and torch.equal(c.cpu().long(), rc)
        R.check(w, rw, rw + 1e-30, n=64)
        assert not bool(w[[0, 3]].any())


@pytest.mark.parametrize("E,groups,top,k", [(8, 1, 1, 2), (16, 1, 1, 5), (32, 8, 4, 6), (64, 1, 1, 6), (64, 8, 3, 8), (128, 4, 2, 8),
                                            (256, 8, 4, 8), (256, 1, 1, 8), (160, 8, 3, 6), (512, 1, 1, 10), (1024, 1, 1, 4)])
@pytest.mark.parametrize("kind", ["normal", "near", "far", "half"])
def test_route_choice_is_the_fp32_formula_of_every_token(E, groups, top, k, kind):
    # every token against the formula in fp32 torch operations (the same roundings): logits of N(0, 1.5); many
    # that differ by a few units in the last place; far ones (tiny scores); bf16 with many equal
    g = torch.Generator(device="cuda").manual_seed(E + k)
    T = 20000 if kind != "normal" else 300000 if E <= 64 else 150000  # more: every warp takes several batches
    l = 1.5 * torch.randn(T, E, device="cuda", generator=g)
    if kind == "near":
        l = torch.randint(-2, 3, (T, E), device="cuda", generator=g) * 0.5 + 1.25  # not 0: its neighbours below are NaN
        l = (l.view(torch.int32) + torch.randint(-3, 4, (T, E), device="cuda", generator=g).int()).view(torch.float32)
    elif kind == "far":
        l = 25 * l - 40
    elif kind == "half":
        l = l.to(BF16)
    for sigmoid in (True, False):
        for bias in (None, 0.1 * torch.randn(E, device="cuda", generator=g)):
            if bias is not None and not sigmoid:
                continue  # the sum's order is the kernel's own
            x = l.float()
            v = 1 / (1 + torch.exp(-x)) if sigmoid else torch.exp(x - x.max(1, keepdim=True).values)
            sel = v if bias is None else v + bias
            if groups > 1:
                best = sel.view(T, groups, -1).sort(dim=2, descending=True).values
                first = (best[:, :, 0] + best[:, :, 1]).sort(dim=1, descending=True, stable=True).indices[:, :top]
                keep = torch.zeros(T, groups, dtype=torch.bool, device="cuda").scatter_(1, first, True)
                sel = torch.where(keep.repeat_interleave(E // groups, 1), sel, -math.inf)
            want = sel.sort(dim=1, descending=True, stable=True).indices[:, :k]
            idx, w, c = run_route(l, bias, sigmoid, groups, top, k, False)
            assert torch.equal(idx.long(), want), (sigmoid, bias is not None, int((idx != want).any(1).sum()))
            assert torch.equal(c.long(), torch.bincount(want.reshape(-1), minlength=E))
            if sigmoid:
                assert torch.equal(w, 2.5 * v.gather(1, want))


def test_route_bias_that_is_not_finite():
    g = gen(4)
    l, b = normal(g, 300, 64), normal(g, 64)
    b[[3, 9]], b[20] = -math.inf, math.inf
    idx, _, _ = run_route(l, b, True, 1, 1, 6, True)
    want = (1 / (1 + torch.exp(-l.cuda())) + b.cuda()).sort(dim=1, descending=True, stable=True).indices[:, :6]
    assert torch.equal(idx.long(), want)
    b[:] = -math.inf
    idx, w, c = run_route(l, b, True, 1, 1, 6, True)
    assert bool((idx == -1).all()) and not bool(w.any()) and not bool(c.any())


def test_route_strided_unaligned_rows_many_tokens_and_reused_workspace():
    g = gen(11)
    big = normal(g, 5000, 301).cuda()
    ws = torch.empty(B.mhc_route_workspace_bytes(256), dtype=torch.uint8, device="cuda")
    B.mhc_workspace_init(ws)
    for at in (0, 1, 3):
        l = big[:, at:at + 256]
        a = run_route(l, None, True, 8, 4, 8, True, ws=ws)
        b = run_route(l.contiguous(), None, True, 8, 4, 8, True, ws=ws)
        assert all(torch.equal(x, y) for x, y in zip(a, b))
        assert int(a[2].sum()) == 5000 * 8
        few = run_route(l[4990:], None, True, 8, 4, 8, True, counts=False)
        assert torch.equal(few[0], a[0][4990:]) and torch.equal(few[1], a[1][4990:])
    idx, w, c = run_route(big[:0, :256], None, True, 1, 1, 8, True, ws=ws)
    assert not bool(c.any())


@pytest.mark.parametrize("E,k,dtype", [(1, 1, F32), (8, 2, F32), (60, 7, BF16), (64, 6, F16), (256, 8, F32), (300, 32, F32),
                                       (1024, 9, BF16)])
@pytest.mark.parametrize("sigmoid,renorm", [(True, True), (True, False), (False, True), (False, False)])
def test_route_grad(E, k, dtype, sigmoid, renorm):
    g = gen(E * k)
    T = 37
    l = normal(g, T, E, std=1.5, dtype=dtype)
    l[5, torch.rand(E, generator=g) < 0.9] = -math.inf
    l[6] = -math.inf
    idx, _, _ = run_route(l, None, sigmoid, 1, 1, k, renorm)
    dw = normal(g, T, k)
    out = torch.full((T, E), 5.0, dtype=dtype, device="cuda")
    B.mhc_route_grad(dev(dw), dev(l), idx, out, score=B.MHC_SCORE_SIGMOID if sigmoid else B.MHC_SCORE_SOFTMAX,
                     renorm=renorm, scale=2.5)
    ref, terms = R.route_grad(dw, l, idx.cpu(), sigmoid, renorm, 2.5)
    R.check(out, ref, terms, n=128, what="dlogits")


@pytest.mark.parametrize("E,k,dtype", [(8, 2, F32), (60, 7, BF16), (256, 8, F32), (300, 32, F32)])
@pytest.mark.parametrize("sigmoid,renorm", [(True, True), (False, False)])
def test_route_grad_of_many_tokens(E, k, dtype, sigmoid, renorm):
    # every token against autograd in 64 bits on the GPU: more tokens than the GPU has warps at a time
    T = 100_003
    g = torch.Generator(device="cuda").manual_seed(E)
    l = (1.5 * torch.randn(T, E, device="cuda", generator=g)).to(dtype)
    idx, _, _ = run_route(l, None, sigmoid, 1, 1, k, renorm)
    dw = torch.randn(T, k, device="cuda", generator=g)
    out = torch.full((T, E), 5.0, dtype=dtype, device="cuda")
    B.mhc_route_grad(dw, l, idx, out, score=int(sigmoid), renorm=renorm, scale=2.5)
    x = l.double().requires_grad_()
    p = (torch.sigmoid(x) if sigmoid else torch.softmax(x, 1)).gather(1, idx.long())
    w = 2.5 * (p / p.sum(1, keepdim=True) if renorm else p)
    (w * dw.double()).sum().backward()
    # the terms of an element are its own and the mean over the k: at most 2.5 * (|dw| + sum |dw|) of its score
    terms = 2.5 * (dw.abs().max(1, keepdim=True).values * (k + 1)).double().expand(T, E)
    terms = terms * (torch.ones_like(x) if renorm else torch.softmax(x, 1)).detach()
    R.check(out, x.grad.cpu(), terms.cpu(), n=32, what="dlogits")


def test_route_grad_skips_foreign_indices_and_takes_strides():
    g = gen(2)
    big = normal(g, 9, 70).cuda()
    l, dst = big[:, 1:51], torch.full((9, 61), 5.0, device="cuda")
    idx = torch.randint(-1, 60, (9, 4), generator=g).int()
    idx[:, 1] = (idx[:, 0] + 1) % 50
    idx[:, 2:] = torch.tensor([-1, 2 ** 31 - 1])
    dw = normal(g, 9, 4)
    B.mhc_route_grad(dev(dw), l, dev(idx), dst[:, 3:53], scale=1.0)
    ref, terms = R.route_grad(dw, l.cpu(), idx, True, True, 1.0)
    R.check(dst[:, 3:53], ref, terms, n=128)
    assert bool((dst[:, :3] == 5).all()) and bool((dst[:, 53:] == 5).all())


def test_route_grad_against_differences():
    g = gen(13)
    T, E, k, h = 4, 12, 3, 1e-5
    l = normal(g, T, E)
    dw = normal(g, T, k)
    for sigmoid in (True, False):
        for renorm in (True, False):
            idx, _, _ = run_route(l, None, sigmoid, 1, 1, k, renorm, scale=1.5)
            out = torch.empty(T, E, device="cuda")
            B.mhc_route_grad(dev(dw), dev(l), idx, out, score=int(sigmoid), renorm=renorm, scale=1.5)

            def loss(x):
                p = R.scores(x, sigmoid)[1].gather(1, idx.cpu().long())
                return (1.5 * (p / p.sum(1, keepdim=True) if renorm else p) * dw.double()).sum()

            for t in range(T):
                for e in range(E):
                    hi, lo = l.double().clone(), l.double().clone()
                    hi[t, e] += h
                    lo[t, e] -= h
                    slope = float((loss(hi) - loss(lo)) / (2 * h))
                    assert abs(slope - float(out[t, e])) < 1e-5 * (1 + abs(slope)), (sigmoid, renorm, t, e)


# ------------------------------------------------- streams, graphs, offsets --
def _chain(stream=None):
    """One pass through all six operators; returns a call and its outputs."""
    g = gen(77)
    T, V, H, E, k = 300, 500, 1056, 64, 4
    ids, table = dev(_ids(g, T, V, "skewed")), normal(g, V, H, dtype=BF16).cuda()
    d = {n: dev(t) for n, t in block_inputs(T, H, BF16, "token", True, True, 78).items()}
    x = torch.empty(T, 1, H, dtype=BF16, device="cuda")
    ro, nm = (torch.empty(T, H, dtype=BF16, device="cuda") for _ in range(2))
    rp, rq, dg = (torch.empty(T, device="cuda") for _ in range(3))
    l = normal(g, T, E).cuda()
    idx, w = torch.empty(T, k, dtype=torch.int32, device="cuda"), torch.empty(T, k, device="cuda")
    c, dl = torch.empty(E, dtype=torch.int32, device="cuda"), torch.empty(T, E, device="cuda")
    dy, dr = (torch.empty(T, H, dtype=BF16, device="cuda") for _ in range(2))
    gp, gq = (torch.empty(H, device="cuda") for _ in range(2))
    dt = torch.empty(V, H, device="cuda")
    wr = torch.zeros(B.mhc_route_workspace_bytes(E), dtype=torch.uint8, device="cuda")
    wb = workspace(B.mhc_block_norm_grad_workspace_bytes(T, H))
    we = workspace(B.mhc_embed_grad_workspace_bytes(T, V, H))

    def call(s=None):
        B.mhc_embed(ids, table, x, stream=s)
        B.mhc_block_norm(d["y"], x[:, 0], d["gamma_post"], d["gate"], d["gamma_pre"], ro, nm, rp, rq,
                         gate_mode=B.MHC_GATE_TOKEN, stream=s)
        B.mhc_route(l, None, idx, w, c, wr, stream=s)
        B.mhc_route_grad(w, l, idx, dl, stream=s)
        B.mhc_block_norm_grad(ro, nm, d["y"], ro, d["gamma_post"], d["gate"], d["gamma_pre"], rp, rq, dy, dr, gp, dg, gq,
                              wb, gate_mode=B.MHC_GATE_TOKEN, stream=s)
        B.mhc_embed_grad(ids, dr, dt, we, stream=s)

    return call, [x, ro, nm, rp, rq, idx, w, c, dl, dy, dr, gp, dg, gq, dt]


def test_operators_on_a_side_stream_and_in_a_graph():
    call, out = _chain()
    call()
    torch.cuda.synchronize()
    want = [t.clone() for t in out]
    s = torch.cuda.Stream()
    for t in out:
        t.zero_()
    s.wait_stream(torch.cuda.current_stream())
    call(s)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(out, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for _ in range(3):
        for t in out:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, want))


def test_first_calls_of_a_process_may_be_captured():
    code = """
import torch
from mhc_residual_seam_gb300 import binding as B
T, V, H, E, k = 3000, 50, 8192, 64, 4
e = lambda *s, t=torch.bfloat16: torch.zeros(*s, dtype=t, device="cuda")
f = torch.float32
ids, table, x, y, w = torch.arange(T, device="cuda") % V, e(V, H) + 1, e(T, H), e(T, H) + 1, e(H) + 1
ro, nm, dy, dr, rp, rq, a, b = e(T, H), e(T, H), e(T, H), e(T, H), e(T, t=f), e(T, t=f), e(H, t=f), e(H, t=f)
l, idx, wt, c = e(T, E, t=f), e(T, k, t=torch.int32), e(T, k, t=f), e(E, t=torch.int32)
dl, dt, wr = e(T, E, t=f), e(V, H, t=f), e(B.mhc_route_workspace_bytes(E), t=torch.uint8)
wb = e(B.mhc_block_norm_grad_workspace_bytes(T, H), t=torch.uint8)
we = e(B.mhc_embed_grad_workspace_bytes(T, V, H), t=torch.uint8)
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    B.mhc_embed(ids, table, x)
    B.mhc_block_norm(y, x, w, None, w, ro, nm, rp, rq)
    B.mhc_route(l, None, idx, wt, c, wr)
    B.mhc_route_grad(wt, l, idx, dl)
    B.mhc_block_norm_grad(ro, nm, y, ro, w, None, w, rp, rq, dy, dr, a, None, b, wb)
    B.mhc_embed_grad(ids, x, dt, we)
g.replay()
torch.cuda.synchronize()
assert bool((dt == T // V).all()) and int(c.sum()) == T * k and bool((ro == 2).all())
"""
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300,
                       cwd=os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
    assert r.returncode == 0, r.stderr[-2000:]


def test_offsets_beyond_32_bits():
    # rows far in a matrix of more than 2^31 elements give what the same rows give alone
    T, H = 270000, 8192
    g = torch.Generator(device="cuda").manual_seed(5)
    big = torch.empty(T, H, dtype=BF16, device="cuda").normal_(generator=g)
    w = torch.ones(H, dtype=BF16, device="cuda")

    def norm(x):
        ro, nm = torch.empty_like(x), torch.empty_like(x)
        rp, rq = (torch.empty(len(x), device="cuda") for _ in range(2))
        B.mhc_block_norm(x, x, w, None, w, ro, nm, rp, rq)
        dy, dr = torch.empty_like(x), torch.empty_like(x)
        a, b = (torch.empty(H, device="cuda") for _ in range(2))
        B.mhc_block_norm_grad(ro, nm, x, ro, w, None, w, rp, rq, dy, dr, a, None, b,
                              workspace(B.mhc_block_norm_grad_workspace_bytes(len(x), H)))
        return ro, nm, rp, rq, dy, dr

    for a, b in zip(norm(big), norm(big[-7:].contiguous())):
        assert torch.equal(a[-7:], b)
    ids = torch.tensor([T - 1, 3, T - 2], device="cuda")
    out = torch.empty(3, H, dtype=BF16, device="cuda")
    B.mhc_embed(ids, big, out)
    assert torch.equal(out, big[ids])
    grad = torch.full((T, H), 2.0, dtype=BF16, device="cuda")
    B.mhc_embed_grad(ids, out, grad, workspace(B.mhc_embed_grad_workspace_bytes(3, T, H)))
    assert torch.equal(grad[ids], out)
    grad[ids] = 0
    assert not bool(grad.any())


def test_route_offsets_beyond_32_bits():
    T, E = 2_200_000, 1024
    l = torch.empty(T, E, dtype=BF16, device="cuda").normal_(generator=torch.Generator(device="cuda").manual_seed(6))
    a, b = run_route(l, None, False, 1, 1, 4, True), run_route(l[-9:].contiguous(), None, False, 1, 1, 4, True)
    assert torch.equal(a[0][-9:], b[0]) and torch.equal(a[1][-9:], b[1]) and int(a[2].sum()) == 4 * T
    d = torch.empty_like(l)
    B.mhc_route_grad(a[1], l, a[0], d, score=B.MHC_SCORE_SOFTMAX)
    e = torch.empty(9, E, dtype=BF16, device="cuda")
    B.mhc_route_grad(b[1], l[-9:], b[0], e, score=B.MHC_SCORE_SOFTMAX)
    assert torch.equal(d[-9:], e)
