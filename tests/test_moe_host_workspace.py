"""Workspaces of the expert layer on the host: the products need none, long
sorts need theirs."""
import pytest

from test_abi_host import POISON as P, qg  # noqa: F401


@pytest.mark.parametrize("m,i,o,e", [(1, 16, 1, 1), (64, 256, 256, 4), (512, 16384, 7168, 1), (65535 * 64, 7168, 2048, 8192),
                                     (0, 0, 0, 0)])
def test_products_need_no_workspace(qg, m, i, o, e):  # noqa: F811
    assert qg.qgemm_e4m3_workspace_bytes(m, i, o, e) == 0


@pytest.mark.parametrize("n,k,e", [(1025, 1, 1), (1 << 20, 8, 256), (2 ** 31 - 1, 1, 8192)])
def test_long_sorts_refuse_less_than_their_workspace(qg, n, k, e):  # noqa: F811
    before, need = qg.qg_launch_count(), qg.qg_moe_sort_workspace_bytes(n, k, e)
    assert need >= 4 * e
    for ws, size in ((0, need), (P, need - 1), (P, 0)):
        assert qg.qg_moe_sort(P, P, P, P, n, k, e, ws, size, stream=0) == qg.QG_EWORKSPACE and str(need) in qg.last_error()
    assert qg.qg_launch_count() == before
