"""Edges of the operators around the seam on the GPU: arguments that have no
effect, choices that only rounding decides, and sums whose order shows."""
import pytest
import torch

from mhc_residual_seam_gb300 import binding as B

from test_block_ops import block_inputs, check_grad, run_block, run_grad

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
