"""Edges of the operators around the seam that need no GPU."""
import pytest
import torch

from mhc_residual_seam_gb300 import binding as B


@pytest.mark.parametrize("H", [8, 64, 256, 264, 512, 520, 1024, 2048, 4096, 5120, 5128, 7168, 8192, 10240, 10248, 16384])
def test_block_norm_grad_workspace_does_not_fall_with_more_tokens(H):
    # a workspace for the most tokens serves fewer: through the steps of the plan (rows of a CTA, CTAs of an SM)
    sizes = [B.mhc_block_norm_grad_workspace_bytes(T, H) for T in range(1, 1300)]
    assert all(a <= b for a, b in zip(sizes, sizes[1:])), next(T for T, (a, b) in enumerate(zip(sizes, sizes[1:])) if a > b)
    far = [B.mhc_block_norm_grad_workspace_bytes(T, H)
           for n in (152, 304, 456, 608, 1216, 2432, 9728) for m in (1, 2, 3, 7, 16, 64, 1000) for T in (n * m - 1, n * m, n * m + 1)]
    assert sizes[-1] >= max(sizes) and max(far) <= B.mhc_block_norm_grad_workspace_bytes(2 ** 31 - 1, H)


@pytest.mark.parametrize("V,H", [(1, 8), (700, 64), (32000, 512), (131072, 5120), (600000, 1024), (2 ** 30, 64)])
def test_embed_grad_workspace_does_not_fall_with_more_tokens(V, H):
    steps = [1, 511, 512, 513, 1023, 1024, 1025, 4095, 4096, 4097, 4609, 65535, 65536, 65537, 65600, 67584, 67585, 100000, 131072,
             131073, 262144, 262145, 10 ** 6, 2 ** 24, 2 ** 30]
    sizes = [B.mhc_embed_grad_workspace_bytes(T, V, H) for T in steps]
    assert all(a <= b for a, b in zip(sizes, sizes[1:])), list(zip(steps, sizes))


def test_the_binding_refuses_calls_without_a_matrix():
    # nothing to take the sizes from: the library's error, not an attribute of None
    w = torch.zeros(64)
    with pytest.raises(B.MhcError) as e:
        B.mhc_block_norm(None, None, None, None, w, None, w, None, w, stream=0)
    assert e.value.code == -1
    with pytest.raises(B.MhcError) as e:
        B.mhc_block_norm_grad(w, w, None, w, None, None, w, None, w, None, None, None, None, w, None, stream=0)
    assert e.value.code == -1
