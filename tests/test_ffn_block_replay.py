"""The serving step of examples/ffn_block.py: its replay is compared in every output, and every workspace's status is read."""
import os
import sys

import pytest
import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

pytestmark = pytest.mark.gpu

OUTPUTS = ("add", "h", "y", "Y", "norm", "residual_out", "pre_out", "post_out", "comb_out")


@pytest.fixture(scope="module")
def M():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import ffn_block
    return ffn_block


@pytest.mark.parametrize("T", [1, 8, 200])
def test_replay_gives_every_output(M, T):
    out = M.serve(T=T)
    for k in OUTPUTS:
        assert torch.equal(out["eager"][k], out["replayed"][k]) and bool(torch.isfinite(out["eager"][k]).all()), k


def test_a_replay_that_writes_nothing_is_seen(M, monkeypatch):
    monkeypatch.setattr(torch.cuda.CUDAGraph, "replay", lambda self: None)
    out = M.serve(T=8)
    for k in OUTPUTS:
        assert not torch.equal(out["eager"][k], out["replayed"][k]), k


def test_every_status_is_read(M, monkeypatch):
    read, check = [], M.B.mhc_check_status
    monkeypatch.setattr(M.B, "mhc_check_status", lambda ws, *a: (read.append(ws.data_ptr()), check(ws, *a)))
    b = M.serve(T=8)["block"]
    assert {b.ws.data_ptr(), b.lora_ws.data_ptr(), b.seam["workspace"].data_ptr()} <= set(read)
