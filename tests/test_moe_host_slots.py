"""The most slots of a token, on the host alone: no pointer is touched and
nothing is launched."""
import pytest

from test_abi_host import POISON as P, qg  # noqa: F401


@pytest.mark.parametrize("k", [2 ** 31 - 9, 2 ** 31 - 8, 2 ** 31 - 1])
def test_slots_of_a_token_that_overflow(qg, k):  # noqa: F811
    """Eight slots go together, so a count of them passes k by up to seven, which has to stay below 2^31."""
    before, t = qg.qg_launch_count(), qg.QG_BF16
    want = qg.QG_OK if k < 2 ** 31 - 8 else qg.QG_EINVAL
    assert qg.qg_moe_dispatch(P, t, None, P, t, 8, P, 0, k, 8, 4, stream=0) == want
    assert qg.qg_moe_dispatch(P, qg.QG_E4M3, P, P, t, 8, P, 0, k, 8, 4, stream=0) == want
    assert qg.qg_moe_combine(P, t, P, t, P, P, 0, k, 8, 4, stream=0) == want
    assert qg.qg_moe_combine_grad(P, P, P, t, P, t, P, P, 0, k, 8, 4, stream=0) == want
    assert qg.qg_launch_count() == before
