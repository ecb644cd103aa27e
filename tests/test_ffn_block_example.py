"""The example that runs the operators inside a block together (examples/ffn_block.py): its
serving step against plain torch and against its own replay, its training gradients against
autograd of a plain 64-bit model, and a training run."""
import os
import sys

import pytest
import torch

import sublayer_case as R

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def M():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import ffn_block
    return ffn_block


@pytest.mark.parametrize("T", [1, 8, 200])
def test_serving_step(M, T):
    out = M.serve(T=T)
    b, e = out["block"], out["eager"]
    for k in ("norm", "residual_out"):
        assert torch.equal(e[k], out["replayed"][k]), k
    d = lambda t: t.double()  # noqa: E731
    x, i = d(out["x"]), out["index"].long()
    has = (i >= 0).double()[:, None]

    def adapters(v, a, w):
        t = torch.einsum("th,trh->tr", v, d(a)[i.clamp_min(0)])
        return 0.5 * has * torch.einsum("tr,tnr->tn", t, d(w)[i.clamp_min(0)])

    near = lambda got, want, n: float((d(got) - want).norm()) <= n * 2.0 ** -9 * float(want.norm())  # noqa: E731
    add = adapters(x, b.up_a, b.up_b)
    assert T == 1 and not has.any() or near(e["add"], add, 1.5)  # one rounding
    gu = x @ d(b.w).t() + d(e["add"])
    g, u = gu.chunk(2, 1)
    h = torch.nn.functional.silu(g) * u
    assert near(e["h"], h, 1.5)
    # the down projection rounds, and so does the sum with the adapters' part
    y = d(e["h"]) @ d(b.w_down).t() + adapters(d(e["h"]), b.down_a, b.down_b)
    assert near(e["y"], y, 3.0)


def plain(p, ids, seed, drop):
    """The example's model in plain 64-bit torch, for autograd."""
    norm = lambda x, w: x / torch.sqrt(x.square().mean(1, keepdim=True) + 1e-6) * w  # noqa: E731
    r = p["table"][ids]
    g, u = (norm(r, p["gamma_in"]) @ p["w"].t()).chunk(2, 1)
    y = (torch.nn.functional.silu(g) * u) @ p["w_down"].t()
    keep = (R.words(*y.shape, *seed) >= int(drop * 2 ** 32 + 0.5)).cuda()
    return norm(r + keep * y / (1 - drop), p["gamma_out"]) @ p["head"]


def test_training_gradients(M):
    p = M.parameters()
    ids = torch.randint(0, 64, (200,), device="cuda", generator=torch.Generator(device="cuda").manual_seed(3))
    seed = (12345, 7)
    loss = torch.nn.functional.cross_entropy(M.model(p, ids, torch.tensor(seed, device="cuda"), 0.1), (ids * 7) % 64)
    loss.backward()
    q = {n: v.detach().double().requires_grad_() for n, v in p.items()}
    want = torch.nn.functional.cross_entropy(plain(q, ids, seed, 0.1), (ids * 7) % 64)
    want.backward()
    assert abs(loss.item() - want.item()) < 0.01 * want.item()
    for n in p:
        a, b = p[n].grad.double(), q[n].grad
        # about twelve bf16 roundings on the way there and back, each 2^-9 of its values with a random sign, twice over
        assert float((a - b).norm()) <= 2 * 12 ** 0.5 * 2.0 ** -9 * float(b.norm()) + 1e-6, (n, float((a - b).norm() / b.norm()))


def test_training_runs(M):
    losses = M.train(steps=20)
    assert len(losses) == 20 and all(x == x and x < 100 for x in losses)
