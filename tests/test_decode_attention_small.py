"""The example's decode loop with budgets below its sinks and recent slots."""
import os
import sys

import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.parametrize("budget,page", [(1, 1), (2, 4), (4, 2), (7, 16)])
def test_small_budgets(budget, page):
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    import decode_attention as ex
    import weight_only_quantized_i4g_gb300 as qg
    g = torch.Generator(device="cuda").manual_seed(budget)
    w_qkv = torch.randn(4 * 64, 128, generator=g, device="cuda") * 128 ** -0.5
    w_o = torch.randn(128, 2 * 64, generator=g, device="cuda") * 128 ** -0.5
    block = ex.AttentionBlock(w_qkv, w_o, 2, 2, 1, 64, budget, page=page)
    for _ in range(60):
        y = block.step(torch.randn(2, 128, generator=g, device="cuda"))
    torch.cuda.synchronize()
    assert bool(torch.isfinite(y).all()) and block.length <= budget + page
    assert qg.qg_device_status() == (0, 0)
