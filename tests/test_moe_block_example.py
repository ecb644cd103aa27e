"""The example that runs the operators together (examples/moe_block.py): its
serving step against plain torch, its training gradients against autograd of a
plain 64-bit model, and a training run."""
import os
import sys

import pytest
import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def M():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import moe_block
    return moe_block


def test_serving_step(M):
    out = M.serve()
    T, k = out["indices"].shape
    assert int(out["counts"].sum()) == T * k
    assert bool((out["indices"] >= 0).all()) and int(out["indices"].max()) < 16
    # renormalised weights of scale 2.5 (k products and sums of fp32)
    assert torch.allclose(out["weights"].sum(1), torch.full((T,), 2.5, device="cuda"), rtol=1e-6)
    # two groups of four experts each
    assert all(len(set(row)) <= 2 for row in (out["indices"] // 4).tolist())
    y = out["y"].double()
    want = y / torch.sqrt(y.square().mean(1, keepdim=True) + 1e-6)
    assert bool(((out["Y"].double() - want).abs() <= 2.0 ** -8 * want.abs() + 1e-6).all())  # one bf16 rounding
    # the next block's input is an RMS norm: mean square 1 up to its bf16 rounding
    assert bool(((out["norm"].double().square().mean(1) - 1).abs() < 2.0 ** -7).all())


def plain(p, ids, k):
    """The example's model in plain 64-bit torch, for autograd."""
    norm = lambda x, w: x / torch.sqrt(x.square().mean(1, keepdim=True) + 1e-6) * w  # noqa: E731
    r = p["table"][ids]
    n = norm(r, p["gamma_in"])
    l = n @ p["w_route"]
    top, idx = l.topk(k, 1)
    w = torch.softmax(top, 1)
    y = torch.zeros_like(n)
    for e in range(l.shape[1]):
        t, j = torch.nonzero(idx == e, as_tuple=True)
        y = y.index_add(0, t, torch.relu(n[t] @ p["w_in"][e]) @ p["w_out"][e] * w[t, j, None])
    return norm(r + p["gate"] * norm(y, p["gamma_post"]), p["gamma_pre"]) @ p["head"]


def test_training_gradients(M):
    p = M.parameters()
    ids = torch.randint(0, 64, (200,), device="cuda", generator=torch.Generator(device="cuda").manual_seed(3))
    loss = torch.nn.functional.cross_entropy(M.model(p, ids), (ids * 7) % 64)
    loss.backward()
    q = {n: v.detach().double().requires_grad_() for n, v in p.items()}
    want = torch.nn.functional.cross_entropy(plain(q, ids, 2), (ids * 7) % 64)
    want.backward()
    assert abs(loss.item() - want.item()) < 1e-4 * want.item()
    for n in p:
        a, b = p[n].grad.double(), q[n].grad
        # fp32 products of up to 128 terms through about six layers (torch's may use TF32-free fp32)
        assert float((a - b).norm()) <= 1e-4 * float(b.norm()), n


def test_training_learns(M):
    losses = M.train(steps=60)
    assert losses[0] > 3.0 and losses[-1] < 0.2 * losses[0]
