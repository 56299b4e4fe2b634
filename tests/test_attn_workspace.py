"""The attention's workspace: what qattn_workspace_bytes() returns for the largest
call of a server covers all of its smaller ones (host only)."""
import pytest

from test_attn_host import P, attn, cache, qg  # noqa: F401

CASES = [  # type, cache heads, query heads, head size, page
    (1, 8, 40, 128, 16), (1, 8, 8, 128, 16), (2, 4, 32, 64, 32), (3, 8, 56, 128, 64), (1, 1, 71, 256, 16), (3, 2, 10, 256, 7),
]
LENGTHS = [1, 17, 130, 300, 520, 700, 1000, 2000, 4000, 4099, 8192, 20000, 131072]


def make(qg, t, heads, dim, page):  # noqa: F811
    return cache(qg, type=t, n_heads=heads, head_dim=dim, page_size=page, token_stride=dim, head_stride=page * dim,
                 page_stride=heads * page * dim)


@pytest.mark.parametrize("t,heads,hq,dim,page", CASES)
@pytest.mark.parametrize("accumulate", [0, 1])
def test_bytes_grow_with_every_size(qg, t, heads, hq, dim, page, accumulate):  # noqa: F811
    c = make(qg, t, heads, dim, page)
    for S in (1, 4, 8):
        last = {}
        for max_len in LENGTHS:
            before = 0
            for n_seq in (*range(1, 40), 64, 76, 77, 152, 153, 300, 2047, 2048, 2049, 5000):
                n = qg.qattn_workspace_bytes(c, n_seq, max_len, S, hq, accumulate)
                assert n >= before and n >= last.get(n_seq, 0), (S, max_len, n_seq)
                if S > 1:
                    assert n >= qg.qattn_workspace_bytes(c, n_seq, max_len, S - 1, hq, accumulate)
                if accumulate:
                    assert n >= qg.qattn_workspace_bytes(c, n_seq, max_len, S, hq, 0)
                before = last[n_seq] = n


@pytest.mark.parametrize("t,heads,hq,dim,page", CASES)
@pytest.mark.parametrize("accumulate", [0, 1])
def test_bytes_of_the_largest_call_serve_all(qg, t, heads, hq, dim, page, accumulate):  # noqa: F811
    """The size is checked before the alignment: a misaligned workspace of enough
    bytes is refused for its alignment (and nothing is launched)."""
    c = make(qg, t, heads, dim, page)
    for most_seq, most_len, most_S in ((64, 700, 1), (19, 4099, 8), (300, 131072, 4)):
        n = qg.qattn_workspace_bytes(c, most_seq, most_len, most_S, hq, accumulate)
        for n_seq in (1, 2, 3, 8, 9, 16, 19, 38, 64, 76, 77, 299, 300):
            for max_len in LENGTHS:
                for S in (1, 3, 4, 8):
                    if n_seq > most_seq or max_len > most_len or S > most_S:
                        continue
                    for acc in {0, accumulate}:
                        rc = attn(qg, c, table_stride=1 << 18, n_seq=n_seq, max_len=max_len, S=S, n_q_heads=hq,
                                  q_type=2 if t == 2 else 1, q_stride=hq * dim, accumulate=acc, ws=P + 16, ws_bytes=n)
                        assert rc == qg.QG_EALIGN, (n_seq, max_len, S, acc, qg.last_error())
