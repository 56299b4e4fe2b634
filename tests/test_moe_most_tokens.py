"""The most tokens a call takes (2^31 - 1): every block is counted."""
import pytest

torch = pytest.importorskip("torch")

from moe_util import DEV  # noqa: E402

pytestmark = pytest.mark.gpu
MOST = 2 ** 31 - 1


@pytest.fixture(scope="module")
def qg():
    import weight_only_quantized_i4g_gb300 as m
    return m


def test_combine_grad_of_the_most_tokens(qg):
    if torch.cuda.mem_get_info()[0] < 40 << 30:
        pytest.skip("needs 40 GB")
    d, y = (torch.empty(MOST, dtype=torch.bfloat16, device=DEV).fill_(v) for v in (3.0, 0.5))
    dy, dw = torch.zeros_like(y), torch.zeros(MOST, dtype=torch.float32, device=DEV)
    qg.check(qg.qg_moe_combine_grad(dy, dw, d, qg.QG_BF16, y, qg.QG_BF16, None, None, MOST, 1, 1, MOST))
    torch.cuda.synchronize()
    for got, want in ((dy, 3.0), (dw, 1.5)):                  # small whole parts: no rounding
        assert all(bool((part == want).all()) for part in got.split(1 << 28))
