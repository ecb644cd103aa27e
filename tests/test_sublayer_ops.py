"""The operators inside a block on the GPU (dropout, the gated projections with
their gradient, adapters of many requests) against plain 64-bit implementations."""
import pytest
import torch

from mhc_residual_seam_gb300 import binding as B

import block_case
import sublayer_case as R

pytestmark = pytest.mark.gpu

BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32


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


def key_of(key, call):
    wrap = lambda v: v - 2 ** 64 if v >= 2 ** 63 else v  # noqa: E731
    return torch.tensor([wrap(key), wrap(call)], device="cuda")


# ----------------------------------------------------------------- dropout --
@pytest.mark.parametrize("T,H,dtype,res,p", [
    (1, 8, BF16, True, 0.5), (3, 40, F16, False, 0.1), (33, 136, F32, True, 0.25), (7, 1032, BF16, False, 0.05),
    (5, 64, F32, False, 0.0), (4, 64, BF16, True, 1.0), (2, 5120, BF16, True, 0.1), (257, 8, F16, True, 0.9)])
def test_dropout(T, H, dtype, res, p):
    g = gen(T + H)
    y, r = normal(g, T, H, dtype=dtype), normal(g, T, H, std=2.0, dtype=dtype) if res else None
    key, call = 0xFEDCBA9876543210, 0x89ABCDEF01234567
    out = torch.full((T, H), 7.0, dtype=dtype, device="cuda")
    B.mhc_dropout(dev(y), out, key_of(key, call), r=dev(r), p=p)
    ref, terms = R.dropout(y, r, p, key, call)
    # the scale's rounding, the product's and the sum's
    block_case.check(out, ref, terms, n=3, what="dropout")
    if not res:
        assert torch.equal(out.cpu() == 0, ref == 0)  # the same mask


def test_dropout_mask_does_not_depend_on_layout():
    T, H = 50, 72
    seed = key_of(11, 3)
    big = normal(gen(1), T, 3 * H, dtype=BF16).cuda()
    y, r = big[:, :H], big[:, 2 * H:]
    want = torch.empty(T, H, dtype=BF16, device="cuda")
    B.mhc_dropout(y.contiguous(), want, seed, r=r.contiguous(), p=0.3)
    holder = torch.full((T, 2 * H), 9.0, dtype=BF16, device="cuda")
    B.mhc_dropout(y, holder[:, H:], seed, r=r, p=0.3)
    assert torch.equal(holder[:, H:], want) and bool((holder[:, :H] == 9).all())
    # in place, on the residual and on y
    a = r.contiguous()
    B.mhc_dropout(y, a, seed, r=a, p=0.3)
    assert torch.equal(a, want)
    b = y.contiguous()
    B.mhc_dropout(b, b, seed, r=r, p=0.3)
    assert torch.equal(b, want)
    # another call's number, another key: other masks
    one = torch.ones(T, H, device="cuda")
    masks = []
    for k in (key_of(11, 3), key_of(11, 4), key_of(12, 3)):
        m = torch.empty_like(one)
        B.mhc_dropout(one, m, k, p=0.5)
        masks.append(m)
    assert not torch.equal(masks[0], masks[1]) and not torch.equal(masks[0], masks[2])


def test_dropout_gradient_is_the_same_call():
    T, H, p = 9, 64, 0.4
    g = gen(3)
    y, d = normal(g, T, H), normal(g, T, H)
    out, dy = torch.empty(T, H, device="cuda"), torch.empty(T, H, device="cuda")
    seed = key_of(5, 6)
    B.mhc_dropout(y.cuda(), out, seed, p=p)
    B.mhc_dropout(d.cuda(), dy, seed, p=p)
    # by differences: out is linear in y
    eps = 0.5
    moved = torch.empty_like(out)
    B.mhc_dropout((y + eps * d).cuda(), moved, seed, p=p)
    # a difference of two rounded values, over eps
    assert torch.allclose((moved - out).double() / eps, dy.double(), rtol=0, atol=float(4 * 2.0 ** -24 * moved.abs().max() / eps))


def test_dropout_leaves_no_trace_of_what_is_dropped():
    T, H = 20, 64
    y = torch.full((T, H), float("nan"), device="cuda")
    r = torch.ones(T, H, device="cuda")
    out = torch.empty(T, H, device="cuda")
    B.mhc_dropout(y, out, key_of(1, 2), r=r, p=0.5)
    keep = (R.words(T, H, 1, 2) >= 2 ** 31).cuda()
    assert torch.equal(torch.isnan(out), keep) and bool((out[~keep] == 1).all())
    B.mhc_dropout(y, out, key_of(1, 2), r=r, p=1.0)
    assert bool((out == 1).all())


def test_dropout_replays_take_the_seed_of_the_moment():
    T, H = 16, 128
    y, out, seed = torch.ones(T, H, device="cuda"), torch.empty(T, H, device="cuda"), key_of(21, 0)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            B.mhc_dropout(y, out, seed, p=0.5)
            seed[1] += 1
    torch.cuda.current_stream().wait_stream(s)
    for call in range(3):
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out.cpu() != 0, R.words(T, H, 21, call) >= 2 ** 31), call


def test_dropout_many_rows():
    # the counter's upper word: element 2^34 is past 32 bits of counters of four
    T, H = 2 ** 21 + 1, 8192
    if torch.cuda.mem_get_info()[0] < 80 << 30:
        pytest.skip("needs 70 GB")
    y = torch.ones(T, H, dtype=BF16, device="cuda")
    B.mhc_dropout(y, y, key_of(3, 4), p=0.5)
    last = [R.philox((i & R.LOW, i >> 32, 4, 0), (3, 0)) for i in range((T - 1) * H // 4, (T - 1) * H // 4 + 16)]
    assert torch.equal(y[-1, :64].cpu() != 0, torch.tensor(last).view(64) >= 2 ** 31)


# ------------------------------------------------------- gated projections --
def workspace(n):
    ws = torch.full((max(n, 16),), 0xA5, dtype=torch.uint8, device="cuda")
    B.mhc_workspace_init(ws)
    return ws


def glu_inputs(T, H, F, dtype, add, seed=0):
    g = gen(seed + T + H + F)
    x, w = normal(g, T, H, dtype=dtype), normal(g, 2 * F, H, std=H ** -0.5, dtype=dtype)
    a = {"none": None, "rows": normal(g, T, 2 * F, std=0.5, dtype=dtype), "bias": normal(g, 1, 2 * F, dtype=dtype)}[add]
    return x, w, a


@pytest.mark.parametrize("T,H,F,dtype,act,add,keep", [
    (1, 8, 8, BF16, "silu", "none", True), (3, 64, 64, F16, "gelu", "rows", True), (16, 72, 40, BF16, "gelu_tanh", "bias", False),
    (17, 136, 136, BF16, "silu", "rows", False), (64, 512, 128, F16, "relu", "none", True), (65, 1032, 72, BF16, "silu", "none", False),
    (127, 200, 256, BF16, "gelu", "bias", True), (128, 320, 264, F16, "silu", "none", True), (129, 64, 1000, BF16, "relu", "rows", True),
    (257, 520, 392, BF16, "gelu_tanh", "none", True), (300, 2056, 136, F16, "silu", "rows", False), (1000, 256, 1368, BF16, "silu", "none", True),
    (1, 5120, 2048, BF16, "silu", "none", False), (4, 2048, 5000, F16, "gelu_tanh", "none", False),
    (33, 1024, 3000, BF16, "silu", "rows", True), (2500, 64, 2048, BF16, "relu", "none", True)])
def test_glu(T, H, F, dtype, act, add, keep):
    x, w, a = glu_inputs(T, H, F, dtype, add)
    ref, terms = R.glu(x, w, a, act)
    ws = workspace(B.mhc_glu_workspace_bytes(T, H, F))
    h = torch.full((T, F), 7.0, dtype=dtype, device="cuda")
    gu = torch.full((T, 2 * F), 7.0, dtype=dtype, device="cuda") if keep else None
    for again in range(2):  # the workspace is as good after a call as before
        B.mhc_glu(dev(x), dev(w), h, ws, add=None if a is None else dev(a).expand(T, 2 * F), gu=gu, act=R.ACTS.index(act))
        B.mhc_check_status(ws)
        block_case.check(h, ref["h"], terms["h"], n=1, what="h")
        if keep:
            block_case.check(gu, ref["gu"], terms["gu"], n=1, what="gu")


def test_glu_strides_and_neighbours():
    T, H, F = 70, 136, 72
    x, w, a = glu_inputs(T, H, F, BF16, "rows")
    want = torch.empty(T, F, dtype=BF16, device="cuda")
    ws = workspace(B.mhc_glu_workspace_bytes(T, H, F))
    B.mhc_glu(dev(x), dev(w), want, ws, add=dev(a))
    wide = torch.full((T, 4, H), float("nan"), dtype=BF16, device="cuda")
    wide[:, 2] = dev(x)
    wide_add = torch.full((T, 2 * F + 8), float("nan"), dtype=BF16, device="cuda")
    wide_add[:, 8:] = dev(a)
    out = torch.full((T + 2, F + 16), 5.0, dtype=BF16, device="cuda")
    B.mhc_glu(wide[:, 2], dev(w), out[1:T + 1, 8:F + 8], ws, add=wide_add[:, 8:])
    assert torch.equal(out[1:T + 1, 8:F + 8], want)
    out[1:T + 1, 8:F + 8] = 5.0
    assert bool((out == 5).all())
    B.mhc_glu(dev(x)[:0], dev(w), want[:0], ws)


@pytest.mark.parametrize("T", [5, 200])
def test_glu_keeps_rows_and_features_apart(T):
    # a NaN in one token's row and an infinity in one feature's weights stay there
    H, F = 72, 200
    x, w, _ = glu_inputs(T, H, F, BF16, "none")
    x[T - 2, 3] = float("nan")
    w[F - 1, 0], w[F + 7, 1] = float("inf"), float("nan")
    h = torch.empty(T, F, dtype=BF16, device="cuda")
    B.mhc_glu(dev(x), dev(w), h, workspace(B.mhc_glu_workspace_bytes(T, H, F)))
    bad = ~torch.isfinite(h).cpu()
    want = torch.zeros(T, F, dtype=torch.bool)
    want[T - 2], want[:, 7] = True, True
    assert torch.equal(bad[:, :F - 1], want[:, :F - 1])


# ----------------------------------------------------- gated gradient --
@pytest.mark.parametrize("T,H,F,dtype,act", [
    (1, 8, 8, BF16, "silu"), (3, 72, 40, F16, "gelu"), (64, 64, 64, BF16, "relu"), (65, 136, 200, BF16, "gelu_tanh"),
    (129, 520, 72, F16, "silu"), (200, 264, 128, BF16, "gelu"), (256, 256, 136, BF16, "silu"), (257, 1032, 264, F16, "relu"),
    (1003, 512, 344, BF16, "gelu"), (700, 64, 1000, BF16, "silu"), (30, 2056, 520, BF16, "gelu_tanh")])
def test_glu_grad(T, H, F, dtype, act):
    x, w, _ = glu_inputs(T, H, F, dtype, "none")
    g = gen(T)
    gu, dh = normal(g, T, 2 * F, std=1.5, dtype=dtype), normal(g, T, F, dtype=dtype)
    ref, terms = R.glu_grad(dh, gu, x, w, act, dtype)
    ws = workspace(B.mhc_glu_workspace_bytes(T, H, F))
    e = lambda *s, t=dtype: torch.full(s, 7.0, dtype=t, device="cuda")  # noqa: E731
    dgu, dx, dw = e(T, 2 * F), e(T, H), e(2 * F, H)
    B.mhc_glu_grad(dev(dh), dev(gu), dev(x), dev(w), dgu, dx, dw, ws, act=R.ACTS.index(act))
    B.mhc_check_status(ws)
    for got, k in ((dgu, "dgu"), (dx, "dx"), (dw, "dw")):
        block_case.check(got, ref[k], terms[k], n=1, what=k)
    # one product alone; 32-bit weights' gradients, added to what is there
    again, dx2 = e(T, 2 * F), e(T, H)
    B.mhc_glu_grad(dev(dh), dev(gu), None, dev(w), again, dx2, None, ws, act=R.ACTS.index(act))
    assert torch.equal(again, dgu)
    block_case.check(dx2, ref["dx"], terms["dx"], n=1, what="dx alone")  # (its sums may be cut at other places)
    old = normal(g, 2 * F, H)
    acc = dev(old)
    B.mhc_glu_grad(dev(dh), dev(gu), dev(x), None, again, None, acc, ws, act=R.ACTS.index(act), accumulate=True)
    block_case.check(acc, ref["dw"] + old.double(), terms["dw"] + old.double().abs(), n=1, what="dw added")
    B.mhc_glu_grad(dev(dh), dev(gu), None, None, again, None, None, ws, act=R.ACTS.index(act))
    assert torch.equal(again, dgu)


def test_glu_grad_of_no_tokens():
    H, F = 64, 72
    ws = workspace(B.mhc_glu_workspace_bytes(1, H, F))
    dw = torch.full((2 * F, H), 3.0, device="cuda")
    z = lambda n: torch.empty(0, n, dtype=BF16, device="cuda")  # noqa: E731
    w = torch.zeros(2 * F, H, dtype=BF16, device="cuda")
    B.mhc_glu_grad(z(F), z(2 * F), z(H), w, z(2 * F), z(H), dw, ws, accumulate=True)
    assert bool((dw == 3).all())
    B.mhc_glu_grad(z(F), z(2 * F), z(H), w, z(2 * F), z(H), dw, ws)
    assert not bool(dw.any())


def test_glu_grad_against_differences():
    # the directional derivative of sum(h * up), from two runs of the forward pass with weights apart by exact steps
    T, H, F = 40, 64, 48
    x, w, _ = glu_inputs(T, H, F, F16, "none")
    ws = workspace(B.mhc_glu_workspace_bytes(T, H, F))
    e = lambda *s: torch.empty(*s, dtype=F16, device="cuda")  # noqa: E731
    h, gu, dgu, dx, dw = e(T, F), e(T, 2 * F), e(T, 2 * F), e(T, H), e(2 * F, H)
    up = normal(gen(8), T, F, dtype=F16)
    B.mhc_glu(dev(x), dev(w), h, ws, gu=gu)
    B.mhc_glu_grad(dev(up), gu, dev(x), dev(w), dgu, dx, dw, ws)
    way = torch.sign(dw.cpu().double())
    step = 2.0 ** -9
    f = []
    for s in (step, -step):
        moved = (w.double() + s * way).to(F16)
        B.mhc_glu(dev(x), dev(moved), h, ws)
        f.append((float((h.cpu().double() * up.double()).sum()), moved.double()))
    want = float((dw.cpu().double() * (f[0][1] - f[1][1])).sum())
    # h's rounding (2^-11 of each term, random signs: five deviations), the gradient's own, and the third derivative
    noise = 5 * 2.0 ** -11 * float((h.cpu().double() * up.double()).square().sum().sqrt()) * 2
    assert abs(f[0][0] - f[1][0] - want) <= noise + 0.01 * abs(want), (f[0][0] - f[1][0], want, noise)


# ---------------------------------------------------------------- adapters --
def lora_inputs(T, H, N, R, n, dtype, order, seed=0):
    g = gen(seed + T + H + N + R)
    x, a, b = normal(g, T, H, dtype=dtype), normal(g, n, R, H, std=H ** -0.5, dtype=dtype), normal(g, n, N, R, std=R ** -0.5, dtype=dtype)
    index = torch.randint(-1, n + 1, (T,), generator=g)
    if order == "runs":
        index = index.sort().values
    if order == "one":
        index[:] = n - 1
    return x, a, b, index.int(), 0.5 + torch.rand(n, generator=g), normal(g, T, N, dtype=dtype)


@pytest.mark.parametrize("T,H,N,rank,n,dtype,order,scaled,based", [
    (1, 8, 8, 8, 1, BF16, "one", False, False), (2, 40, 72, 8, 3, F16, "any", True, True), (17, 136, 64, 16, 4, BF16, "any", True, True),
    (16, 1032, 200, 24, 2, BF16, "one", True, False), (33, 264, 136, 32, 40, F16, "any", False, True), (64, 520, 256, 16, 32, BF16, "any", True, True),
    (64, 512, 320, 64, 5, BF16, "runs", True, True), (65, 72, 1000, 40, 3, F16, "one", True, False), (130, 2056, 72, 64, 7, F16, "runs", True, True),
    (200, 320, 264, 128, 3, BF16, "any", False, False), (100, 64, 520, 256, 2, F16, "any", True, True), (300, 5120, 64, 16, 9, BF16, "runs", True, True),
    (63, 96, 8, 72, 70, BF16, "any", True, True)])
def test_lora(T, H, N, rank, n, dtype, order, scaled, based):
    x, a, b, index, scale, base = lora_inputs(T, H, N, rank, n, dtype, order)
    scale, base = scale if scaled else None, base if based else None
    ref, terms = R.lora(x, a, b, index, scale, base)
    ws = workspace(B.mhc_lora_workspace_bytes(T, rank))
    out = torch.full((T, N), 7.0, dtype=dtype, device="cuda")
    args = (dev(x), dev(a), dev(b), dev(index))
    B.mhc_lora(*args, out, ws, scale=dev(scale), base=dev(base))
    block_case.check(out, ref, terms, n=1, what="lora")
    none = ((index < 0) | (index >= n)).cuda()
    assert torch.equal(out[none], dev(base)[none] if based else torch.zeros_like(out[none]))
    if based:  # in place
        again = dev(base).clone()
        B.mhc_lora(*args, again, ws, scale=dev(scale), base=again)
        assert torch.equal(again, out)


def test_lora_strides_and_neighbours():
    T, H, N, r, n = 70, 136, 72, 16, 4
    x, a, b, index, scale, base = (dev(t) for t in lora_inputs(T, H, N, r, n, BF16, "any"))
    ws = workspace(B.mhc_lora_workspace_bytes(T, r))
    want = torch.empty(T, N, dtype=BF16, device="cuda")
    B.mhc_lora(x, a, b, index, want, ws, scale=scale, base=base)
    wide = torch.full((T, 4, H), float("nan"), dtype=BF16, device="cuda")
    wide[:, 1] = x
    holder = torch.full((T + 2, N + 16), 5.0, dtype=BF16, device="cuda")
    inner = holder[1:T + 1, 8:N + 8]
    inner.copy_(base)
    B.mhc_lora(wide[:, 1], a, b, index, inner, ws, scale=scale, base=inner)
    assert torch.equal(inner, want)
    inner.fill_(5.0)
    assert bool((holder == 5).all())
    B.mhc_lora(x[:0], a, b, index[:0], want[:0], ws, scale=scale)


def test_lora_keeps_tokens_and_adapters_apart():
    # values of every size: fp16 sums past 65504, tiny rows, a NaN row, an infinite one, a broken adapter
    T, H, N, r, n = 40, 256, 64, 16, 3
    x, a, b, index, _, _ = lora_inputs(T, H, N, r, n, F16, "any")
    index = index.clamp(0, n - 1)
    x[3], x[4] = 60000.0, 2.0 ** -20
    a[:] = a.abs()
    b *= 2.0 ** -8
    ref, terms = R.lora(x, a, b, index, None, None)
    x[5, 7], x[6, 8] = float("nan"), float("inf")
    index[7] = 2
    a[2, 3, 4] = float("nan")
    out = torch.empty(T, N, dtype=F16, device="cuda")
    ws = workspace(B.mhc_lora_workspace_bytes(T, r))
    B.mhc_lora(dev(x), dev(a), dev(b), dev(index), out, ws)
    fine = index != 2
    fine[5] = fine[6] = fine[7] = False
    block_case.check(out[fine.cuda()], ref[fine], terms[fine], n=1)
    assert not bool(torch.isfinite(out[5]).any()) and not bool(torch.isfinite(out[6]).any())
    assert bool(torch.isnan(out[(index == 2).cuda()]).all())


def test_lora_results_do_not_depend_on_neighbours_order():
    # tokens of the same adapter in another order in the batch give the same rows
    T, H, N, r, n = 64, 512, 128, 32, 8
    x, a, b, index, scale, base = (dev(t) for t in lora_inputs(T, H, N, r, n, BF16, "any"))
    ws = workspace(B.mhc_lora_workspace_bytes(T, r))
    out, moved = torch.empty(T, N, dtype=BF16, device="cuda"), torch.empty(T, N, dtype=BF16, device="cuda")
    B.mhc_lora(x, a, b, index, out, ws, scale=scale, base=base)
    p = torch.randperm(T, generator=gen(2)).cuda()
    B.mhc_lora(x[p], a, b, index[p], moved, ws, scale=scale, base=base[p])
    assert torch.equal(moved, out[p])


def test_glu_calls_of_other_sizes_share_a_workspace():
    sizes = [(5, 512, 1000), (128, 1024, 200), (1, 72, 3000), (64, 4096, 136), (200, 64, 72), (3, 2048, 640)]
    ws = workspace(max(B.mhc_glu_workspace_bytes(*s) for s in sizes))
    for again in range(2):
        for T, H, F in sizes:
            x, w, _ = glu_inputs(T, H, F, BF16, "none")
            ref, terms = R.glu(x, w, None, "silu")
            h = torch.empty(T, F, dtype=BF16, device="cuda")
            B.mhc_glu(dev(x), dev(w), h, ws)
            block_case.check(h, ref["h"], terms["h"], n=1)
    B.mhc_check_status(ws)


def test_glu_of_a_few_tokens_repeats_bit_for_bit():
    # the sums of runs that share a tile do not depend on which of them ends last
    T, H, F = 9, 5120, 2000
    x, w, _ = (dev(t) if t is not None else None for t in glu_inputs(T, H, F, BF16, "none"))
    ws = workspace(B.mhc_glu_workspace_bytes(T, H, F))
    want = torch.empty(T, F, dtype=BF16, device="cuda")
    B.mhc_glu(x, w, want, ws)
    for _ in range(50):
        h = torch.empty_like(want)
        B.mhc_glu(x, w, h, ws)
        assert torch.equal(h, want)


@pytest.mark.parametrize("T,H,N,rank,n,order", [(65, 64, 72, 8, 100, "any"), (1024, 72, 8, 16, 3, "any"), (1025, 40, 64, 8, 2, "one"),
                                                (2100, 64, 136, 24, 600, "any"), (3000, 136, 64, 40, 5, "runs"), (2048, 8, 8, 8, 1, "any"), (500, 72, 1000, 64, 7, "runs"), (1500, 64, 264, 96, 40, "any"), (130, 40, 128, 200, 3, "runs")])
def test_lora_of_many_tokens(T, H, N, rank, n, order):
    x, a, b, index, scale, base = lora_inputs(T, H, N, rank, n, BF16, order)
    out = torch.full((T, N), 7.0, dtype=BF16, device="cuda")
    ws = workspace(B.mhc_lora_workspace_bytes(T, rank))
    B.mhc_lora(dev(x), dev(a), dev(b), dev(index), out, ws, scale=dev(scale), base=dev(base))
    some = torch.cat([torch.arange(min(T, 70)), torch.randint(0, T, (150,), generator=gen(1)), torch.arange(T - 40, T)]).unique()
    ref, terms = R.lora(x[some], a, b, index[some], scale, base[some])
    block_case.check(out[some.cuda()], ref, terms, n=1, what="lora")
    # every token, against the same call token by token in other company
    p = torch.randperm(T, generator=gen(2)).cuda()
    moved = torch.empty_like(out)
    B.mhc_lora(dev(x)[p], dev(a), dev(b), dev(index)[p], moved, ws, scale=dev(scale), base=dev(base)[p])
    assert bool(((moved.double() - out[p].double()).abs() <= 2.0 ** -7 * out[p].double().abs() + 1e-4).all())


# ------------------------------------------------- sizes that cut tiles along k --
# (whole rounds and a rest; a few tiles with long sums; both products of the gradient at once)
@pytest.mark.parametrize("T,H,F,dtype", [(1100, 2048, 5000, BF16), (256, 4096, 10000, F16), (130, 8192, 264, BF16), (2304, 1536, 4224, BF16),
                                         (16384, 64, 72, F16), (129, 16384, 8, BF16), (128, 16384, 24, F16), (2, 72, 40000, BF16)])
def test_glu_of_larger_sizes(T, H, F, dtype):
    x, w, a = (dev(t) for t in glu_inputs(T, H, F, dtype, "rows"))
    ref, terms = R.glu(x, w, a, "silu")
    ws = workspace(B.mhc_glu_workspace_bytes(T, H, F))
    want = None
    for _ in range(3):
        h, gu = torch.full((T, F), 7.0, dtype=dtype, device="cuda"), torch.full((T, 2 * F), 7.0, dtype=dtype, device="cuda")
        B.mhc_glu(x, w, h, ws, add=a, gu=gu)
        if want is None:
            want = (h, gu)
            block_case.check(h, ref["h"].cpu(), terms["h"].cpu(), n=1, what="h")
            block_case.check(gu, ref["gu"].cpu(), terms["gu"].cpu(), n=1, what="gu")
        assert torch.equal(h, want[0]) and torch.equal(gu, want[1])  # the same bits whatever the timing
    B.mhc_check_status(ws)


@pytest.mark.parametrize("T,H,F,dtype", [(3000, 520, 2000, BF16), (128, 512, 20000, F16), (20000, 72, 64, BF16), (1024, 1024, 4096, BF16),
                                         (700, 2920, 1000, F16), (5, 40, 16384, BF16)])
def test_glu_grad_of_larger_sizes(T, H, F, dtype):
    x, w, _ = (None if t is None else dev(t) for t in glu_inputs(T, H, F, dtype, "none"))
    g = gen(T)
    gu, dh = dev(normal(g, T, 2 * F, dtype=dtype)), dev(normal(g, T, F, std=0.1, dtype=dtype))
    ref, terms = R.glu_grad(dh, gu, x, w, "silu", dtype)
    ws = workspace(B.mhc_glu_workspace_bytes(T, H, F))
    want = None
    for _ in range(3):
        e = lambda *s: torch.full(s, 7.0, dtype=dtype, device="cuda")  # noqa: E731
        out = {"dgu": e(T, 2 * F), "dx": e(T, H), "dw": e(2 * F, H)}
        B.mhc_glu_grad(dh, gu, x, w, out["dgu"], out["dx"], out["dw"], ws)
        if want is None:
            want = out
            for k in out:
                block_case.check(out[k], ref[k].cpu(), terms[k].cpu(), n=1, what=k)
        assert all(torch.equal(out[k], want[k]) for k in out)
    acc = torch.ones(2 * F, H, device="cuda")
    B.mhc_glu_grad(dh, gu, x, w, out["dgu"], out["dx"], acc, ws, accumulate=True)
    block_case.check(acc, ref["dw"].cpu() + 1, terms["dw"].cpu() + 1, n=1, what="dw added")
    B.mhc_check_status(ws)


# --------------------------------------------------------- streams and graphs --
def test_two_streams_with_workspaces_of_their_own():
    sizes = [(64, 1024, 2000), (300, 512, 1368)]
    jobs = []
    for T, H, F in sizes:
        x, w, _ = glu_inputs(T, H, F, BF16, "none")
        lx, la, lb, li, ls, lbase = (dev(t) for t in lora_inputs(T, H, 264, 16, 5, BF16, "any"))
        jobs.append({"x": dev(x), "w": dev(w), "ws": workspace(B.mhc_glu_workspace_bytes(T, H, F)), "stream": torch.cuda.Stream(),
                     "h": torch.empty(T, F, dtype=BF16, device="cuda"), "lora": (lx, la, lb, li), "scale": ls, "base": lbase,
                     "out": torch.empty_like(lbase), "lws": workspace(B.mhc_lora_workspace_bytes(T, 16))})
    for j in jobs:
        B.mhc_glu(j["x"], j["w"], j["h"], j["ws"])
        B.mhc_lora(*j["lora"], j["out"], j["lws"], scale=j["scale"], base=j["base"])
        j["want"] = (j["h"].clone(), j["out"].clone())
    torch.cuda.synchronize()
    for _ in range(20):
        for j in jobs:
            B.mhc_glu(j["x"], j["w"], j["h"], j["ws"], stream=j["stream"])
            B.mhc_lora(*j["lora"], j["out"], j["lws"], scale=j["scale"], base=j["base"], stream=j["stream"])
    torch.cuda.synchronize()
    for j in jobs:
        assert torch.equal(j["h"], j["want"][0]) and torch.equal(j["out"], j["want"][1])


FIRST = """
import torch
from mhc_residual_seam_gb300 import binding as B
T, H, F = %d, 512, 1000
n = lambda *s: torch.randn(*s, device="cuda").bfloat16()
x, w, dh, a, b = n(T, H), n(2 * F, H), n(T, F), n(3, 16, H), n(3, 2 * F, 16)
e = lambda *s: torch.zeros(*s, device="cuda", dtype=torch.bfloat16)
add, h, gu, dgu, dx, dw, out = e(T, 2 * F), e(T, F), e(T, 2 * F), e(T, 2 * F), e(T, H), e(2 * F, H), e(T, H)
index, seed = torch.arange(T, device="cuda").int() %% 4 - 1, torch.tensor([1, 2], device="cuda")
ws = torch.zeros(B.mhc_glu_workspace_bytes(T, H, F), device="cuda", dtype=torch.uint8)
lws = torch.zeros(B.mhc_lora_workspace_bytes(T, 16), device="cuda", dtype=torch.uint8)
def calls():
    B.mhc_lora(x, a, b, index, add, lws)
    B.mhc_glu(x, w, h, ws, add=add, gu=gu)
    B.mhc_glu_grad(dh, gu, x, w, dgu, dx, dw, ws)
    B.mhc_dropout(dx, out, seed, r=x, p=0.5)
s = torch.cuda.Stream()
s.wait_stream(torch.cuda.current_stream())
with torch.cuda.stream(s):
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        calls()  # the first calls of the process are captured
torch.cuda.current_stream().wait_stream(s)
for t in (add, h, gu, dgu, dx, dw, out):
    t.zero_()
g.replay()
torch.cuda.synchronize()
got = [t.clone() for t in (add, h, gu, dgu, dx, dw, out)]
g.replay()
torch.cuda.synchronize()
assert all(torch.equal(p, q) for p, q in zip(got, (add, h, gu, dgu, dx, dw, out)))
calls()
torch.cuda.synchronize()
assert all(torch.equal(p, q) for p, q in zip(got, (add, h, gu, dgu, dx, dw, out)))
assert all(bool(torch.isfinite(t).all()) and bool(t.any()) for t in got)
B.mhc_check_status(ws)
print("fine")
"""


@pytest.mark.parametrize("T", [7, 300])
def test_first_calls_under_capture(T):
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", FIRST % T], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "fine" in r.stdout, r.stderr[-2000:]


def test_weights_written_just_before_the_call():
    # the call starts beside the end of the kernel that writes its weights (here a gradient), and reads what that one wrote
    T, H, F = 600, 1024, 2048
    x, w, _ = (None if t is None else dev(t) for t in glu_inputs(T, H, F, BF16, "none"))
    few = dev(normal(gen(6), 5, H, dtype=BF16))
    ws, ws2 = workspace(B.mhc_glu_workspace_bytes(T, H, F)), workspace(B.mhc_glu_workspace_bytes(T, H, F))
    e = lambda *s: torch.empty(*s, dtype=BF16, device="cuda")  # noqa: E731
    gu, dgu, dw, h, big = dev(normal(gen(7), T, 2 * F, dtype=BF16)), e(T, 2 * F), e(2 * F, H), e(5, F), e(T, F)
    for i in range(6):
        dh = dev(normal(gen(20 + i), T, F, std=0.02, dtype=BF16))
        dw.fill_(float("nan"))
        B.mhc_glu_grad(dh, gu, x, None, dgu, None, dw, ws)
        B.mhc_glu(few, dw, h, ws2)
        B.mhc_glu(x, dw, big, ws2)
        got = (h.clone(), big.clone())
        torch.cuda.synchronize()
        B.mhc_glu(few, dw, h, ws2)
        torch.cuda.synchronize()
        B.mhc_glu(x, dw, big, ws2)
        assert bool(torch.isfinite(got[0]).all()) and torch.equal(got[0], h) and torch.equal(got[1], big)
    # and an adapter's result is the projections' addend, the projections' output the adapter's input
    a, b, index = dev(normal(gen(8), 3, 16, H, dtype=BF16)), dev(normal(gen(9), 3, 2 * F, 16, dtype=BF16)), (torch.arange(T) % 4 - 1).int().cuda()
    add, lws = e(T, 2 * F), workspace(B.mhc_lora_workspace_bytes(T, 16))
    for rows in (5, 64, 65, T):
        want = None
        for _ in range(4):
            add.fill_(float("nan"))
            B.mhc_lora(x[:rows], a, b, index[:rows], add[:rows], lws)
            B.mhc_glu(x[:rows], w, big[:rows], ws, add=add[:rows])
            if want is None:
                torch.cuda.synchronize()
                B.mhc_glu(x[:rows], w, big[:rows], ws, add=add[:rows])
                want = big[:rows].clone()
            assert torch.equal(big[:rows], want) and bool(torch.isfinite(want).all())


# --------------------------------------------------------- offsets past 32 bits --
def test_offsets_past_32_bits():
    if torch.cuda.mem_get_info()[0] < 60 << 30:
        pytest.skip("needs 50 GB")
    g = torch.Generator(device="cuda").manual_seed(1)
    rand = lambda *s, std=1.0: torch.empty(*s, device="cuda", dtype=BF16).normal_(0, std, generator=g)  # noqa: E731
    T, H, F = 135001, 64, 8192  # T * 2F is past 2^31
    x, w, add = rand(T, H), rand(2 * F, H, std=0.125), rand(T, 2 * F)
    h, gu = torch.empty(T, F, dtype=BF16, device="cuda"), torch.empty(T, 2 * F, dtype=BF16, device="cuda")
    ws = workspace(B.mhc_glu_workspace_bytes(T, H, F))
    B.mhc_glu(x, w, h, ws, add=add, gu=gu)
    rows = torch.tensor([0, 65535, 131071, 131072, T - 129, T - 1], device="cuda")
    ref, terms = R.glu(x[rows], w, add[rows], "silu")
    block_case.check(h[rows], ref["h"].cpu(), terms["h"].cpu(), n=1, what="h")
    block_case.check(gu[rows], ref["gu"].cpu(), terms["gu"].cpu(), n=1, what="gu")
    dh, dgu, dx = h, add, torch.empty(T, H, dtype=BF16, device="cuda")
    B.mhc_glu_grad(dh, gu, None, w, dgu, dx, None, ws)
    ref, terms = R.glu_grad(dh[rows], gu[rows], x[rows], w, "silu", BF16)
    block_case.check(dgu[rows], ref["dgu"].cpu(), terms["dgu"].cpu(), n=1, what="dgu")
    block_case.check(dx[rows], ref["dx"].cpu(), terms["dx"].cpu(), n=1, what="dx")
    del h, gu, dh, dgu, add
    N = 2 * F
    for rank in (16, 64):
        a, b = rand(3, rank, H, std=0.125), rand(3, N, rank, std=0.25)
        base, out = rand(T, N), torch.empty(T, N, dtype=BF16, device="cuda")
        index = (torch.arange(T, device="cuda") % 4 - 1).int()
        B.mhc_lora(x, a, b, index, out, workspace(B.mhc_lora_workspace_bytes(T, rank)), base=base)
        ref, terms = R.lora(x[rows].cpu(), a.cpu(), b.cpu(), index[rows].cpu(), None, base[rows].cpu())
        block_case.check(out[rows], ref, terms, n=1, what="lora")
        del base, out


def test_a_reported_wait_is_an_error_once():
    ws = workspace(B.mhc_glu_workspace_bytes(4, 64, 64))
    ws[:4].view(torch.int32).fill_(2)  # as a wait that ran out leaves it
    with pytest.raises(B.MhcError) as e:
        B.mhc_check_status(ws)
    assert e.value.code == -7
    B.mhc_check_status(ws)


def test_chains_of_calls_read_what_the_last_one_wrote():
    # each call starts beside the end of the one before it; every output is the next one's input
    T, H, F = 700, 512, 1024
    x, w, _ = (None if t is None else dev(t) for t in glu_inputs(T, H, F, BF16, "none"))
    w2, seed = dev(normal(gen(3), 2 * F, F, std=F ** -0.5, dtype=BF16)), key_of(1, 2)
    a, b, index = dev(normal(gen(4), 2, 64, F, std=0.05, dtype=BF16)), dev(normal(gen(5), 2, F, 64, std=0.1, dtype=BF16)), (torch.arange(T) % 3 - 1).int().cuda()
    ws, lws = workspace(B.mhc_glu_workspace_bytes(T, F, F)), workspace(B.mhc_lora_workspace_bytes(T, 64))
    e = lambda *s: torch.empty(*s, dtype=BF16, device="cuda")  # noqa: E731
    gu, h, drop, more, h2, dgu, dx, last = e(T, 2 * F), e(T, F), e(T, F), e(T, F), e(T, F), e(T, 2 * F), e(T, H), e(T, H)
    outs = (gu, h, drop, more, h2, dgu, dx, last)

    def chain(sync):
        wait = torch.cuda.synchronize if sync else (lambda: None)
        for t in outs:
            t.fill_(float("nan"))
        B.mhc_glu(x, w, h, ws, gu=gu); wait()  # noqa: E702
        B.mhc_dropout(h, drop, seed, p=0.25); wait()  # noqa: E702
        B.mhc_lora(drop, a, b, index, more, lws, base=drop); wait()  # noqa: E702
        B.mhc_glu(more, w2, h2, ws); wait()  # noqa: E702
        B.mhc_glu_grad(h2, gu, x, w, dgu, dx, None, ws); wait()  # noqa: E702
        B.mhc_dropout(dx, last, seed, r=x, p=0.5); wait()  # noqa: E702
        torch.cuda.synchronize()
        return [t.clone() for t in outs]

    want = chain(True)
    assert all(bool(torch.isfinite(t).all()) for t in want)
    for _ in range(20):
        assert all(torch.equal(p, q) for p, q in zip(chain(False), want))
