"""Sizes that the attention counts in 31 bits: large batches of long capacities
are split over launches, and only a sequence that is too long by itself is
refused."""
import pytest

from test_attn_host import P, attn, cache, qg  # noqa: F401


def make(qg, heads, page, dim=128):  # noqa: F811
    return cache(qg, n_heads=heads, page_size=page, head_dim=dim, token_stride=dim, head_stride=page * dim,
                 page_stride=heads * page * dim)


@pytest.mark.parametrize("heads,hq,page,n_seq,max_len,S", [
    (8, 64, 16, 256, 131072, 8), (8, 64, 1, 128, 131072, 1), (8, 64, 1, 5000, 1 << 20, 8), (8, 64, 16, 2, 1 << 30, 8),
    (1, 8, 1, 100, (1 << 30) - 2, 1), (64, 1024, 16, 3000, 131072, 8), (8, 8, 3, 100000, 1 << 20, 1)])
def test_calls_that_fit_are_not_refused(qg, heads, hq, page, n_seq, max_len, S):  # noqa: F811
    """The sizes are checked before the workspace's alignment (and nothing is launched)."""
    c = make(qg, heads, page)
    kw = dict(n_seq=n_seq, max_len=max_len, S=S, n_q_heads=hq, q_stride=hq * 128, table_stride=-(-max_len // page))
    assert qg.qattn_workspace_bytes(c, n_seq, max_len, S, hq) > 0
    assert attn(qg, c, ws=P + 16, **kw) == qg.QG_EALIGN, qg.last_error()


@pytest.mark.parametrize("heads,hq,page,n_seq,max_len,S", [
    (64, 64, 1, 1, 1 << 30, 1), (1, 8, 1, 1, 1 << 30, 1), (8, 1024, 16, 1, 1 << 30, 8), (8, 64, 16, 1 << 25, 1000, 8)])
def test_sequences_too_long_by_themselves_are_refused(qg, heads, hq, page, n_seq, max_len, S):  # noqa: F811
    c = make(qg, heads, page)
    assert qg.qattn_workspace_bytes(c, n_seq, max_len, S, hq) == 0
    assert attn(qg, c, n_seq=n_seq, max_len=max_len, S=S, n_q_heads=hq, q_stride=hq * 128,
                table_stride=-(-max_len // page)) == qg.QG_EINVAL
    assert "overflow" in qg.last_error()


@pytest.mark.gpu
@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
def test_batches_split_by_their_capacity(qg, kv):  # noqa: F811
    """A capacity of 2^30 slots: every sequence is a launch of its own."""
    torch = pytest.importorskip("torch")
    from attn_util import DEV, Paged, check_attention
    from test_attn_paged import queries
    pc = Paged(qg, [700, 0, 45, 130], 8, 64, kv, page=64, seed=31).fill()
    wide = torch.full((4, 1 << 24), -1, dtype=torch.int32, device=DEV)
    wide[:, :pc.width] = pc.table
    pc.table, pc.width = wide, 1 << 24
    check_attention(pc, queries(pc, 4, 2, 16, kv), 2, 16, 0.125, max_len=1 << 30)


@pytest.mark.gpu
@pytest.mark.parametrize("page", [(1 << 31) - 1, (1 << 31) - 14])
def test_one_page_of_the_largest_size(qg, page):  # noqa: F811
    """A cache without pages to speak of: k and v share one pool of 2^31 slots."""
    torch = pytest.importorskip("torch")
    if torch.cuda.mem_get_info()[0] < 45 << 30:
        pytest.skip("needs 45 GB")
    dim, n = 8, 1000
    pool = torch.empty(1, 1, page, dim, dtype=torch.bfloat16, device="cuda")
    pool[:, :, :n + 16] = torch.randn(n + 16, dim, device="cuda").bfloat16()
    c = qg.kv_cache(pool, pool)
    q = torch.randn(1, 2 * dim, device="cuda").bfloat16()
    o = torch.empty(1, 2, dim, device="cuda")
    table, lens = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in ([[0]], [n]))
    for max_len in (n, 1 << 30):
        size = qg.qattn_workspace_bytes(c, 1, max_len, 1, 2)
        ws = torch.empty(max(size, 1), dtype=torch.uint8, device="cuda")
        o.fill_(float("nan"))
        qg.check(qg.qattn_paged(c, table, 1, lens, 1, max_len, o, qg.QG_F32, None, q, qg.QG_BF16, 2 * dim, 1, 2, 0.3,
                                0, ws, size))
        torch.cuda.synchronize()
        assert qg.qg_device_status() == (0, 0)
        x = pool[0, 0, :n].double()
        want = torch.softmax(q.view(2, dim).double() @ x.T * 0.3, -1) @ x
        assert float((o[0].double() - want).abs().max()) < 1e-4
