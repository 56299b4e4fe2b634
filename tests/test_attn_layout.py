"""The attention kernels' index arithmetic, checked on the CPU by a host program
built from their headers (tests/attn_layout_check.cu): exact divisions, the
swizzled places of a step's chunks against the copies' rule, bank conflicts of
the fragment reads, shared-memory budgets of every instantiation, and 3000
splits of ragged batches over blocks and groups of warps (every step once, in
order; spans of shared segments)."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
PKG = os.path.join(ROOT, "weight_only_quantized_i4g_gb300")
NVCC = os.environ.get("NVCC", "/usr/local/cuda/bin/nvcc")


def test_attention_index_arithmetic(tmp_path):
    if not (os.path.exists(NVCC) or shutil.which("nvcc")):
        pytest.skip("nvcc not available")
    exe = str(tmp_path / "attn_layout_check")
    r = subprocess.run([NVCC, "-O1", "-std=c++17", "--expt-relaxed-constexpr", "-gencode",
                        "arch=compute_103a,code=sm_103a", "-I", os.path.join(PKG, "csrc"), "-I",
                        os.path.join(ROOT, "include"), "-o", exe, os.path.join(ROOT, "tests", "attn_layout_check.cu"),
                        "-L", PKG, "-l:libqgemv.so", "-Xlinker", "-rpath," + PKG],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stdout + r.stderr
    r = subprocess.run([exe], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.rstrip().endswith("ok"), r.stdout[-3000:]
