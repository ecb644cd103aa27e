"""Edges of the operators around the seam on the GPU: arguments that have no
effect, choices that only rounding decides, and sums whose order shows."""
import math

import pytest
import torch

from mhc_residual_seam_gb300 import binding as B

import block_case as R
from test_block_ops import block_inputs, check_grad, dev, gen, normal, run_block, run_grad, run_route

pytestmark = pytest.mark.gpu

BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    B.lib()


# ------------------------------------------------------------- block norms --
@pytest.mark.parametrize("T,H,dtype", [(40, 640, BF16), (3, 264, F32), (700, 1032, F16)])
@pytest.mark.parametrize("scale", [0.75, -2.0, 0.0])
def test_the_norm_without_y_takes_no_residual_scale(T, H, dtype, scale):
    # norm = r / rms(r) * gamma_pre, whatever res_scale: neither it nor its gradient is scaled
    d = block_inputs(T, H, dtype, "none", False, True, 21, y=False)
    o, one = run_block(d, "none", scale=scale), run_block(d, "none", scale=1.0)
    assert torch.equal(o["norm"], one["norm"]) and torch.equal(o["rstd_pre"], one["rstd_pre"])
    check_grad(d, "none", o, run_grad(d, "none", o, scale=scale), scale=1.0)


def test_the_gradient_without_y_against_differences_and_autograd():
    T, H, scale, eps, h = 3, 24, 0.75, 1e-6, 1e-4
    d = block_inputs(T, H, F32, "none", False, True, 31, y=False)
    o = run_block(d, "none", scale, eps)
    q = run_grad(d, "none", o, scale)

    def loss(r, w):  # r goes on as it is, and through the norm
        norm = r / torch.sqrt(r.square().mean(1, keepdim=True) + eps) * w
        return (r * d["dr_out"].double()).sum() + (norm * d["dnorm"].double()).sum()

    r, w = d["r"].double().requires_grad_(), d["gamma_pre"].double().requires_grad_()
    loss(r, w).backward()
    for got, leaf in (("dr", r), ("dgamma_pre", w)):
        flat = q[got].cpu().double().reshape(-1)
        # sums of at most H products of fp32 roundings
        assert bool(((flat - leaf.grad.reshape(-1)).abs() < 1e-4 * (1 + leaf.grad.reshape(-1).abs())).all()), got
        for at in range(0, flat.numel(), max(1, flat.numel() // 5)):
            v = {"dr": [r.detach().clone(), w.detach()], "dgamma_pre": [r.detach(), w.detach().clone()]}[got]
            x = v[0] if got == "dr" else v[1]
            x.reshape(-1)[at] += h
            up = loss(*v)
            x.reshape(-1)[at] -= 2 * h
            slope = float((up - loss(*v)) / (2 * h))
            assert abs(slope - float(flat[at])) < 2e-4 * (1 + abs(slope)), (got, at)


# ----------------------------------------------------------------- routing --
def clear_choice(l, bias, groups, top, k, gap):
    """The choice of softmax + bias in 64 bits, and the rows where every comparison that decides is wider than `gap`."""
    T, E = l.shape
    sel = torch.softmax(l.double(), 1) + bias.double()
    sel = torch.where(l > -math.inf, sel, -math.inf)
    clear = torch.ones(T, dtype=torch.bool, device=l.device)
    if groups > 1:
        best = sel.view(T, groups, -1).sort(dim=2, descending=True).values
        val, order = (best[:, :, 0] + best[:, :, 1]).sort(dim=1, descending=True)
        clear &= (val[:, top - 1] - val[:, top] > gap)
        keep = torch.zeros(T, groups, dtype=torch.bool, device=l.device).scatter_(1, order[:, :top], True)
        sel = torch.where(keep.repeat_interleave(E // groups, 1), sel, -math.inf)
    val, idx = sel.sort(dim=1, descending=True)
    n = min(k, E - 1)
    clear &= ((val[:, :n] - val[:, 1:n + 1]) > gap).all(1)
    return idx[:, :k], clear


# fp32 scores of softmax + bias: exp (2 ulp), a sum of E terms (32 in a lane, then 5 levels), a division and the
# bias's addition leave each at most 45 * 2^-24 of itself off, and the scores of a row add up to one; sums of two
# such choices, up to 3 in size, are rounded twice more
GAP = 5e-6


@pytest.mark.parametrize("E,groups,top,k", [(64, 1, 1, 6), (8, 1, 1, 2), (32, 8, 3, 4), (128, 4, 2, 8), (256, 8, 4, 8), (256, 1, 1, 8),
                                            (160, 8, 3, 6), (512, 1, 1, 10), (1024, 1, 1, 4)])
@pytest.mark.parametrize("offset", [0.0, 1e3, 1e5, 1e6])
def test_softmax_with_a_bias_does_not_depend_on_a_common_offset(E, groups, top, k, offset):
    g = torch.Generator(device="cuda").manual_seed(E + k)
    T = 100000
    l = 1.5 * torch.randn(T, E, device="cuda", generator=g) + offset
    bias = 0.1 * torch.randn(E, device="cuda", generator=g)
    want, clear = clear_choice(l, bias, groups, top, k, GAP)
    assert float(clear.double().mean()) > 0.7
    idx, w, c = run_route(l, bias, False, groups, top, k, True)
    assert torch.equal(idx.long()[clear], want[clear]), int((idx[clear] != want[clear]).any(1).sum())
    assert torch.equal(c.long(), torch.bincount(idx.long().reshape(-1), minlength=E))


@pytest.mark.parametrize("E,groups", [(8, 1), (64, 1), (64, 8), (256, 1), (256, 8)])
def test_softmax_with_a_bias_chooses_between_near_scores_of_large_logits(E, groups):
    # two experts in play, 3 apart; the second one's bias makes up for it but for a little, for every maximum
    T = 20000
    m = torch.arange(T, device="cuda") * 0.25 + 16  # a multiple of 1/4: the difference is exact
    a, b = 1, E - 1
    p = 1 / (1 + math.exp(-3.0))
    for little in (6e-6, 1e-5, 2e-5, 4e-5, -6e-6, -1e-5, -2e-5, -4e-5):
        l = torch.full((T, E), -math.inf, device="cuda")
        l[:, a], l[:, b] = m, m - 3
        bias = torch.zeros(E, device="cuda")
        bias[b] = 2 * p - 1 - little
        want, clear = clear_choice(l, bias, 1, 1, 1, 5.5e-6)
        assert bool(clear.all()) and bool((want == (a if little > 0 else b)).all())
        idx, _, _ = run_route(l, bias, False, groups, 1, 1, False)
        assert torch.equal(idx.long(), want), (little, int((idx != want).sum()))


@pytest.mark.parametrize("top", [3e9, 1e12, 1e30, 3e38])
def test_softmax_with_a_bias_of_very_large_logits(top):
    # the best expert's share is 1 and the others' 0
    l = torch.zeros(1000, 64, device="cuda")
    at = torch.arange(1000, device="cuda") % 64
    l[torch.arange(1000, device="cuda"), at] = top * (1 - torch.arange(1000, device="cuda") * 1e-4)
    bias = 0.25 - torch.arange(64, device="cuda") / 512.0
    idx, w, _ = run_route(l, bias, False, 1, 1, 2, False, scale=1.0)
    assert torch.equal(idx[:, 0].long(), at) and torch.equal(idx[:, 1].long(), (at == 0).long())
    assert bool((w[:, 0] == 1).all()) and bool((w[:, 1] == 0).all())


@pytest.mark.parametrize("E,groups", [(32, 4), (64, 8), (256, 8)])
@pytest.mark.parametrize("live,top", [(3, 2), (4, 2), (4, 3)])
def test_equal_groups_of_different_experts_go_to_the_lowest(E, groups, live, top):
    # saturated sigmoids (scores of 1): the groups' sums of two are equal to the bit, their members are not
    per = E // groups
    pairs = [(0.25, 0.5), (0.125, 0.625), (0.4375, 0.3125), (0.1875, 0.5625)][:live]
    l, bias = torch.full((100, E), -math.inf), torch.zeros(E)
    for n, (x, y) in enumerate(pairs):
        e = (groups - live + n) * per
        l[:, e:e + 2] = 40.0
        bias[e], bias[e + 1] = x, y
    idx, w, c = run_route(l, bias, True, groups, top, 2 * top, False, scale=1.0)
    first = [(groups - live + n) * per + i for n in range(top) for i in range(2)]
    want = sorted(first, key=lambda e: -float(bias[e]))
    assert bool((idx.cpu() == torch.tensor(want, dtype=torch.int32)).all()), (idx[0].tolist(), want)
    assert bool((w == 1).all()) and int(c.sum()) == 100 * 2 * top


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("above", [64.0, 96.0, 120.0, 1000.0])
def test_renormalised_softmax_of_experts_far_below_one_that_is_kept_out(above, dtype):
    # the weights are the chosen scores' ratio, which does not depend on the row's maximum
    T, E, k = 200, 64, 4
    l = normal(gen(17), T, E).to(dtype)
    bias = torch.arange(E) / 64.0  # the scores of the others are 0 beside it
    bias[5] = -math.inf
    l[:, 5] = above + l.float().max().ceil()
    idx, w, _ = run_route(l, bias, False, 1, 1, k, True, scale=2.5)
    assert bool((idx.cpu() == torch.tensor([63, 62, 61, 60], dtype=torch.int32)).all())
    want = 2.5 * torch.softmax(l.double()[:, [63, 62, 61, 60]], 1)
    R.check(w, want, want, n=64, what="weights")
    # and the gradient is that of these weights
    dw = normal(gen(18), T, k)
    out = torch.empty(T, E, dtype=dtype, device="cuda")
    B.mhc_route_grad(dev(dw), dev(l), idx, out, score=B.MHC_SCORE_SOFTMAX, scale=2.5)
    ref, terms = R.route_grad(dw, torch.where(torch.arange(E) == 5, -math.inf, l.float()), idx.cpu(), False, True, 2.5)
    R.check(out, ref, terms, n=128, what="dlogits")


@pytest.mark.parametrize("renorm", [False, True])
def test_the_gradient_of_saturated_sigmoids(renorm):
    # s' = s (1 - s), with 1 - s = 1 / (1 + exp(l)) for large logits, where 1 - s from s would be 0
    T, E, k = 400, 32, 4
    g = gen(23)
    l = 8 + 72 * torch.rand(T, E, generator=g)
    idx, _, _ = run_route(l, None, True, 1, 1, k, renorm)
    dw = normal(g, T, k)
    out = torch.empty(T, E, device="cuda")
    B.mhc_route_grad(dev(dw), dev(l), idx, out, renorm=renorm, scale=2.5)
    x = l.double().gather(1, idx.cpu().long())
    s, rest = 1 / (1 + torch.exp(-x)), 1 / (1 + torch.exp(x))
    if renorm:
        q = s / s.sum(1, keepdim=True)
        mean = (q * dw.double()).sum(1, keepdim=True)
        d, terms = q * (dw.double() - mean) * rest, q * (dw.double().abs() + (q * dw.double().abs()).sum(1, keepdim=True)) * rest
    else:
        d = terms = dw.double() * s * rest
    # exp twice 2 ulp, the products, sums of four
    R.check(out.cpu().gather(1, idx.cpu().long()), 2.5 * d, 2.5 * terms.abs(), n=32, what="dlogits")


@pytest.mark.parametrize("E,sigmoid,renorm", [(8, True, False), (256, True, False), (64, False, False)])
def test_an_expert_named_often_adds_up_in_slot_order(E, sigmoid, renorm):
    T, k = 500, 8
    g = gen(29)
    idx = torch.randint(0, 3, (T, k), generator=g).int()  # each several times
    idx[::7, 2] = -1
    idx[::5] = E - 1
    dw = (2.0 ** torch.randint(0, 30, (T, k), generator=g)) * torch.randint(-1, 2, (T, k), generator=g)
    l = torch.zeros(T, E)
    outs = []
    for _ in range(3):
        out = torch.empty(T, E, device="cuda")
        B.mhc_route_grad(dev(dw), dev(l), dev(idx), out, score=int(sigmoid), renorm=renorm, scale=1.0)
        outs.append(out.cpu())
    assert all(torch.equal(outs[0], o) for o in outs)
    up = torch.zeros(T, E)
    for j in range(k):  # one rounding per addition
        t = torch.nonzero(idx[:, j] >= 0)[:, 0]
        up[t, idx[t, j].long()] += dw[t, j]
    if sigmoid:
        want = 0.25 * up
    else:  # every score is 1 / E, a power of two; the mean is a sum over 32 lanes, halves first
        mean = torch.zeros(T, 32)
        mean[:, :k] = torch.where(idx >= 0, dw / E, 0.0)
        while mean.shape[1] > 1:
            mean = mean[:, :mean.shape[1] // 2] + mean[:, mean.shape[1] // 2:]
        want = (up - mean) / E
    assert torch.equal(outs[0], want), int((outs[0] != want).any(1).sum())


@pytest.mark.parametrize("E,groups,top,k", [(8, 1, 1, 2), (33, 1, 1, 5), (64, 8, 3, 6), (64, 1, 1, 9), (128, 4, 2, 8), (256, 8, 4, 8),
                                            (256, 1, 1, 12), (384, 1, 1, 4), (512, 8, 3, 2), (1024, 16, 14, 2)])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_a_bias_that_is_not_finite_changes_nothing_but_its_expert(E, groups, top, k, dtype):
    # an expert without a finite bias makes the router choose every token from the exact scores; on an expert that
    # is never chosen the results are the same bits as from the estimates, whatever the sizes of logits and biases
    g = torch.Generator(device="cuda").manual_seed(E + k)
    for n, (std, offset, size) in enumerate([(1.0, 0.0, 0.1), (1.5, 1e6, 0.1), (0.01, 300.0, 1e-4), (40.0, -60.0, 1.0), (3.0, 5e3, 30.0),
                                             (1e-3, 1e9, 1e-6), (0.5, 80.0, 1e3)]):
        l = (std * torch.randn(20000, E, device="cuda", generator=g) + offset).to(dtype)
        if n % 2:
            l[torch.rand(l.shape, device="cuda", generator=g) < 0.3] = -math.inf
        if n % 3 == 2:
            l[torch.rand(l.shape, device="cuda", generator=g) < 0.01] = math.inf
        dead = (7 * n + 3) % E
        l[:, dead] = -math.inf
        bias = size * torch.randn(E, device="cuda", generator=g)
        other = bias.clone()
        other[dead] = -math.inf
        for sigmoid in (True, False):
            a, b = (run_route(l, x, sigmoid, groups, top, k, n % 2 == 0) for x in (bias, other))
            assert all(torch.equal(x, y) for x, y in zip(a, b)), (n, sigmoid, int((a[0] != b[0]).any(1).sum()))
