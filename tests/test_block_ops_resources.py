"""Kernels of the operators around the seam by the assembler's own report (nvcc
-Xptxas -v, no GPU): no variant is compiled that no plan takes, and spills stay
where the kernels' comments say they are."""
import os
import re
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "mhc_residual_seam_gb300", "csrc")
NVCC = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"

pytestmark = pytest.mark.skipif(not os.path.exists(NVCC), reason="nvcc not available")


def kernels(src, out):
    r = subprocess.run([NVCC, "-gencode", "arch=compute_103a,code=sm_103a", "-O3", "-std=c++17", "-I",
                        os.path.join(ROOT, "include"), "-Xptxas", "-v", "-c", os.path.join(CSRC, src), "-o", str(out)],
                       capture_output=True, text=True, timeout=600)
    assert r.returncode == 0, r.stderr[-2000:]
    found, name = {}, None
    for line in r.stderr.splitlines():
        m = re.search(r"Compiling entry function '(\w+)'", line)
        if m:
            name = m.group(1)
        m = re.search(r"(\d+) bytes spill stores", line)
        if m and name:
            found[name] = int(m.group(1))
    return found


def arguments(name):
    return [int(x) for x in re.findall(r"L[ib](\d+)E", name)]


def test_block_norm_variants(tmp_path):
    found = kernels("mhc_block_norm.cu", tmp_path / "norm.o")
    forward = {n: arguments(n) for n in found if "block_norm_kernel" in n}
    grad = {n: arguments(n) for n in found if "block_norm_grad_kernel" in n}
    assert forward and grad
    # forward (groups, a warp per row, rows ahead, no tests): a row always fits, so rows are always fetched ahead
    assert all(a[2] > 0 for a in forward.values())
    # gradient (groups, a warp per row, wide, rows ahead, no tests): a warp has one group of columns; only wide fp32
    # rows do not fit; 16-bit rows of one warp always fit four times
    assert not [n for n, a in grad.items() if a[1] and a[0] == 2]
    assert all(a[2] and "If" in n for n, a in grad.items() if a[3] == 0)
    assert all(a[3] == 4 for n, a in grad.items() if a[1] and "If" not in n)
    assert len(forward) == 2 * 9 + 9 and len(grad) == 2 * 10 + 10
    for n, a in grad.items():
        assert found[n] <= (400 if a[2] else 64), (n, found[n])
    assert all(found[n] <= 64 for n in forward)


def test_other_operators_hardly_spill(tmp_path):
    for src in ("mhc_route.cu", "mhc_embed.cu", "mhc_embed_grad.cu"):
        for n, spill in kernels(src, tmp_path / "o.o").items():
            assert spill <= 32, (n, spill)
