"""Which kernels the parametrised tests of the e4m3 products reach: every tile
width, every split of K and the many-token kernel, in the tests against 64 bits
and in the exact ones, so that a changed constant of the choice cannot leave a
kernel without a test unseen."""
import os
import shutil
import subprocess

import pytest

torch = pytest.importorskip("torch")

import test_gemm_e4m3  # noqa: E402
import test_gemm_e4m3_sums  # noqa: E402
from moe_util import U, blocks, guarded, product, unharmed  # noqa: E402
from test_gemm_e4m3 import call, codes, qg, scales  # noqa: E402, F401

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
PKG = os.path.join(ROOT, "weight_only_quantized_i4g_gb300")
NVCC = os.environ.get("NVCC", "/usr/local/cuda/bin/nvcc")


@pytest.fixture(scope="module")
def chosen(tmp_path_factory):
    """plans of (rows, inner, outer, experts)"""
    if not (os.path.exists(NVCC) or shutil.which("nvcc")):
        pytest.skip("nvcc not available")
    exe = str(tmp_path_factory.mktemp("plans") / "dump")
    r = subprocess.run([NVCC, "-std=c++17", "--expt-relaxed-constexpr", "-gencode", "arch=compute_103a,code=sm_103a",
                        "-I", os.path.join(PKG, "csrc"), "-o", exe, os.path.join(ROOT, "tests", "e4m3_plan_dump.cu"),
                        "-L", PKG, "-l:libqgemv.so", "-Xlinker", "-rpath," + PKG], capture_output=True, text=True)
    assert r.returncode == 0, r.stdout + r.stderr

    def plans(sizes):
        r = subprocess.run([exe], input="".join("%d %d %d %d\n" % s for s in sizes), capture_output=True, text=True, timeout=120)
        assert r.returncode == 0, r.stderr
        return dict(zip(sizes, r.stdout.splitlines(), strict=True))
    return plans


def sizes(dense, groups, extra):
    return [(m, i, o, 1) for m, i, o in dense] + [(sum(c) + extra, i, o, len(c)) for c, i, o in groups if i % 16 == 0]


# splits of K by two and four that no other test reaches
MORE = [(40, 1920, 130), (50, 2048, 300), (64, 2064, 129), (100, 5120, 7680), (128, 1536, 500), (300, 1024, 130)]


@pytest.mark.parametrize("m,i,o", MORE)
def test_more_splits(qg, m, i, o):  # noqa: F811
    """Against 64 bits, within the f32 additions that test_gemm_e4m3_sums counts."""
    x, w = codes((m, i), 1, 60.0), codes((1, o, i), 2, 60.0)
    xs, ws = scales((m, blocks(i)), 3, False), scales((1, blocks(o), blocks(i)), 4, False)
    y = guarded((m, o), torch.float32)
    qg.check(call(qg, y, x, xs, w, ws))
    want, mag = product(x, xs, w, ws, [0, m])
    assert bool(((y.double() - want).abs() <= (265 + blocks(i)) * U * mag).all()) and unharmed(y)


def test_products_reach_every_kernel(chosen):
    got = chosen(sizes(test_gemm_e4m3.DENSE + MORE, test_gemm_e4m3.GROUPS, 3))
    print(got)
    assert set(got.values()) >= {"many"} | {f"few {bt} {c}" for bt in (32, 64, 128) for c in (1, 2, 4, 8)}


def test_exact_sums_reach_every_kernel(chosen):
    got = chosen(sizes([d for d in test_gemm_e4m3_sums.DENSE if d[1] % 16 == 0], test_gemm_e4m3_sums.GROUPS, 0))
    print(got)
    assert {v.rsplit(" ", 1)[0] for v in got.values()} >= {"many", "few 32", "few 64", "few 128"}
