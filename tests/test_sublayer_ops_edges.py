"""The operators inside a block where they can go wrong: no adapters at all."""
import pytest
import torch

from mhc_residual_seam_gb300 import binding as B

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
