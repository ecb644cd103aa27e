"""Kernels of the operators inside a block by the assembler's own report (nvcc
-Xptxas -v, no GPU): which variants are compiled, their registers and spills."""
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
            found[name] = {"spill": 0, "regs": 0}
        m = re.search(r"(\d+) bytes spill stores", line)
        if m and name:
            found[name]["spill"] = int(m.group(1))
        m = re.search(r"Used (\d+) registers", line)
        if m and name:
            found[name]["regs"] = int(m.group(1))
    return found


def test_products(tmp_path):
    glu, grad = kernels("mhc_glu.cu", tmp_path / "g.o"), kernels("mhc_glu_grad.cu", tmp_path / "d.o")
    # two tile shapes and the form for a few tokens, two types; the gradient's one or two products
    assert sum("product_kernel" in n for n in glu) == 4 and sum("glu_few_kernel" in n for n in glu) == 2
    assert sum("product_kernel" in n for n in grad) == 8 and sum("act_grad" in n for n in grad) == 8
    for n, k in {**glu, **grad}.items():
        assert k["spill"] == 0 and k["regs"] <= 168, (n, k)  # 384 threads a CTA, one CTA an SM


def test_dropout_and_adapters(tmp_path):
    drop, lora = kernels("mhc_dropout.cu", tmp_path / "p.o"), kernels("mhc_lora.cu", tmp_path / "l.o")
    # residual or not, dense or strided; fp32 has one item a step only
    assert len(drop) == 2 * 2 * (2 + 2 + 1) and all(k["spill"] == 0 and k["regs"] <= 64 for k in drop.values())
    # ranks up to 8, 16, 32, 64 and in passes of 128; up to 16, 32, 64 and 128 with and without a base; tcgen05 with and without
    assert sum("shrink" in n for n in lora) == 2 * 5 and sum("expand" in n for n in lora) == 2 * 8
    assert sum("wide" in n for n in lora) == 2 * 2 and sum("plan" in n for n in lora) == 1
    for n, k in lora.items():
        assert k["spill"] <= 96, (n, k)
