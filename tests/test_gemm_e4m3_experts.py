"""e4m3 products over more experts than one launch's tables hold: against 64
bits with most experts empty, tables that decrease across the launches' borders,
and the launches counted (the tensor-core kernels take 1024 experts each, the
general one any number)."""
import pytest

torch = pytest.importorskip("torch")

from moe_util import DTYPES, blocks, guarded, ints, product, unharmed  # noqa: E402
from test_gemm_e4m3 import as_f32, call, codes, held, qg, scales  # noqa: E402, F401
from test_gemm_e4m3_offsets import check_table  # noqa: E402

pytestmark = pytest.mark.gpu


def some_rows(experts, filled, most, seed):
    g = torch.Generator().manual_seed(seed)
    counts = torch.zeros(experts, dtype=torch.long)
    counts[torch.randperm(experts, generator=g)[:filled]] = torch.randint(1, most + 1, (filled,), generator=g)
    return counts.tolist()


# 1024 experts, one and two launches' borders, the most experts; rows on both sides of the borders and at the last expert
CASES = [(1024, {0: 3, 1023: 5}, 256, 136), (1025, {0: 3, 1023: 5, 1024: 70}, 256, 136), (1025, {1024: 1}, 128, 128),
         (2048, {1023: 2, 1024: 9, 2047: 4}, 272, 72), (3000, 60, 256, 136), (3000, 900, 128, 40), (8192, {0: 1, 5000: 40, 8191: 33}, 128, 24),
         (2000, {7: 2000, 1500: 3001}, 128, 264), (1025, {3: 5, 1024: 2}, 135, 40)]


@pytest.mark.parametrize("experts,rows,i,o", CASES)
@pytest.mark.parametrize("power,yt", [(False, "f32"), (True, "bf16")])
def test_many_experts(qg, experts, rows, i, o, power, yt):  # noqa: F811
    counts = [rows.get(e, 0) for e in range(experts)] if isinstance(rows, dict) else some_rows(experts, rows, 6, experts)
    bounds = [2]                                              # two rows before the first expert, three behind the last
    for c in counts:
        bounds.append(bounds[-1] + c)
    n = bounds[-1]
    x, w = codes((n + 3, i), 1, 20.0), codes((experts, o, i), 2, 20.0)
    xs, ws = scales((n + 3, blocks(i)), 3, False), scales((experts, blocks(o), blocks(i)), 4, power)
    y = guarded((n + 3, o), DTYPES[yt])
    before = qg.qg_launch_count()
    qg.check(call(qg, y, x, xs, w, ws, ints(bounds)))
    assert qg.qg_launch_count() - before == (-(-experts // 1024) if i % 16 == 0 else 1)
    want, mag = product(x, xs, w, as_f32(ws), bounds)
    assert held(y[2:n], want[2:n], mag[2:n], yt)
    assert bool((y[:2] == 7).all()) and bool((y[n:] == 7).all()) and unharmed(y)
    assert qg.qg_device_status() == (qg.QG_OK, qg.QG_OK)


@pytest.mark.parametrize("i", [128, 135])
@pytest.mark.parametrize("where", [5, 1000, 1023, 1024, 1025, 1400])
def test_tables_that_decrease_across_launches(qg, i, where):  # noqa: F811
    """The offset `where` jumps to 90 of 100 rows; the ones behind it go on from below, so only rows past 90 are left."""
    table = [min(e // 8, 60) for e in range(1501)]
    table[where] = 90
    table[-1] = 97
    check_table(qg, table, 100, i, 40)


@pytest.mark.parametrize("experts,i", [(1, 256), (3, 256), (3, 135)])
def test_without_a_workspace(qg, experts, i):  # noqa: F811
    """Its size is 0 for every call: NULL will do."""
    x, w = codes((30, i), 1, 20.0), codes((experts, 40, i), 2, 20.0)
    xs, ws = scales((30, blocks(i)), 3, False), scales((experts, 1, blocks(i)), 4, False)
    bounds = [30 * e // experts for e in range(experts + 1)]
    y = guarded((30, 40), DTYPES["f32"])
    if experts == 1:
        qg.check(qg.qgemm_e4m3(qg.QG_FMT_FP8B128, y, qg.QG_F32, x, xs, w, ws, 30, i, 40, None, 0))
    else:
        qg.check(qg.qgemm_e4m3_moe(qg.QG_FMT_FP8B128, y, qg.QG_F32, x, xs, w, ws, ints(bounds), experts, 30, i, 40, None, 0))
    want, mag = product(x, xs, w, ws, bounds)
    assert held(y, want, mag, "f32") and unharmed(y)


def test_captured_and_replayed_with_other_offsets(qg):  # noqa: F811
    """Two launches in a graph, rows before, across and behind the border between them."""
    experts, m, i, o = 1500, 200, 256, 136
    x, w = codes((m, i), 1, 20.0), codes((experts, o, i), 2, 20.0)
    xs, ws = scales((m, blocks(i)), 3, False), scales((experts, blocks(o), blocks(i)), 4, False)
    off, y = ints([0] * (experts + 1)), torch.zeros(m, o, device=x.device)
    qg.check(call(qg, y, x, xs, w, ws, off))
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        qg.check(qg.qgemm_e4m3_moe(qg.QG_FMT_FP8B128, y, qg.QG_F32, x, xs, w, ws, off, experts, m, i, o))
    for seed, rows in enumerate(({0: 200}, {1499: 150}, {1023: 90, 1024: 110}, {5: 60, 1200: 70}, {})):
        counts = [rows.get(e, 0) for e in range(experts)]
        bounds = [0]
        for c in counts:
            bounds.append(bounds[-1] + c)
        off.copy_(ints(bounds))
        y.fill_(7)
        graph.replay()
        torch.cuda.synchronize()
        n = bounds[-1]
        want, mag = product(x, xs, w, ws, bounds)
        assert held(y[:n], want[:n], mag[:n], "f32") and bool((y[n:] == 7).all()), seed
