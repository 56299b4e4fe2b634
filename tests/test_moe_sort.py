"""Slots sorted by expert on the GPU against lists: equal, in every element,
for one slot and many, one expert and thousands, experts without a slot, slots
without an expert."""
import pytest

torch = pytest.importorskip("torch")

from moe_util import DEV, ints, routing, sorted_slots  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def qg():
    import weight_only_quantized_i4g_gb300 as m
    return m


def sort(qg, ids, experts, order=True, stream=None):
    n, k = len(ids), len(ids[0]) if ids else 1
    off = torch.full((experts + 1 + 8,), -7, dtype=torch.int32, device=DEV)
    od = torch.full((n * k + 8,), -7, dtype=torch.int32, device=DEV)
    pl = torch.full((n * k + 8,), -7, dtype=torch.int32, device=DEV)
    wb = qg.qg_moe_sort_workspace_bytes(n, k, experts)
    ws = torch.full((max(wb, 1),), 0xFF, dtype=torch.uint8, device=DEV)
    qg.check(qg.qg_moe_sort(off, od if order else None, pl, ints(ids) if ids else None, n, k, experts, ws, wb, stream))
    torch.cuda.synchronize()
    return off.tolist(), od.tolist(), pl.tolist()


@pytest.mark.parametrize("tokens,k,experts,away", [
    (1, 1, 1, 0.0), (1, 8, 64, 0.0), (3, 2, 5, 0.0), (8, 8, 128, 0.0), (31, 1, 4, 0.0), (33, 3, 7, 0.5), (64, 1, 1, 0.0),
    (257, 6, 60, 0.1), (1000, 8, 256, 0.0), (1025, 1, 8192, 0.0), (1024, 8, 2, 0.9), (4099, 5, 33, 0.2), (5, 40, 8, 0.0),
    (9000, 2, 1000, 0.0), (30011, 8, 256, 0.1), (70001, 1, 3, 0.0), (20000, 4, 8192, 0.3), (300, 4, 16, 1.0)])
def test_sort(qg, tokens, k, experts, away):
    ids = routing(tokens, k, experts, tokens + k, away)
    offsets, order, place = sorted_slots(ids, experts)
    off, od, pl = sort(qg, ids, experts)
    assert off == offsets + [-7] * 8
    assert pl == place + [-7] * 8
    assert od == order + [-7] * (tokens * k - len(order) + 8)       # behind the last row nothing is written


def test_no_order_wanted(qg):
    ids = routing(100, 4, 16, 3)
    off, od, pl = sort(qg, ids, 16, order=False)
    offsets, _, place = sorted_slots(ids, 16)
    assert off[:17] == offsets and pl[:400] == place and od == [-7] * 408


def test_no_tokens(qg):
    off = torch.full((9,), -7, dtype=torch.int32, device=DEV)
    qg.check(qg.qg_moe_sort(off, None, None, None, 0, 4, 8))
    assert off.tolist() == [0] * 9


def test_one_expert_takes_all(qg):
    ids = [[5]] * 40000
    off, od, pl = sort(qg, ids, 9)
    assert off[:10] == [0] * 6 + [40000] * 4
    assert od[:40000] == list(range(40000)) and pl[:40000] == list(range(40000))


def test_other_stream_and_repeats(qg):
    ids = routing(5000, 8, 64, 11, 0.1)
    first = sort(qg, ids, 64)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        for _ in range(5):
            assert sort(qg, ids, 64) == first
