"""An empty batch: no sequences and no tokens (host only)."""
from test_attn_host import append, attn, evict, qg  # noqa: F401


def test_an_empty_batch_is_no_error(qg):  # noqa: F811
    n0 = qg.qg_launch_count()
    assert append(qg, T=0, n_seq=0, table=None, seq=None, slot=None) == qg.QG_OK
    assert attn(qg, n_seq=0) == qg.QG_OK and evict(qg, n_seq=0) == qg.QG_OK
    assert qg.qg_launch_count() == n0
    for kw in (dict(n_seq=0, T=1), dict(n_seq=-1, T=0)):
        assert append(qg, **kw) == qg.QG_EINVAL and "n_seq" in qg.last_error()
