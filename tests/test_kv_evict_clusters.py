"""Eviction where several blocks share a head and where a block's work outgrows
its registers and its shared memory: windows without a middle to choose from,
more than 1024 slots a warp, more keys than a block holds."""
import math

import pytest

torch = pytest.importorskip("torch")

from attn_util import DEV, Paged, ints  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def qg():
    import weight_only_quantized_i4g_gb300 as m
    return m


def definition(w, n, budget, sinks, recent):
    """Kept slots of every head, w f32 [heads, n] on the CPU: protected ends,
    then a stable sort (NaN above +inf, ties to the lower slot)."""
    heads = w.shape[0]
    if n <= budget:
        return torch.arange(n).repeat(heads, 1)
    mid = w[:, sinks:n - recent].double()
    by_value = torch.sort(torch.where(mid.isnan(), math.inf, mid), dim=-1, descending=True, stable=True).indices
    nan_first = torch.sort(mid.isnan().gather(1, by_value).byte(), dim=-1, descending=True, stable=True).indices
    best = by_value.gather(1, nan_first)[:, :budget - sinks - recent]
    ends = torch.cat([torch.arange(sinks), torch.arange(n - recent, n)]).repeat(heads, 1)
    return torch.cat([ends, best + sinks], -1).sort(-1).values


def run(qg, lens, heads, budget, sinks, recent, kv="e4m3", page=16, kind="ties", max_len=None):
    kept_pages = [-(-min(n, budget) // page) for n in lens]
    pc = Paged(qg, lens, heads, 16, kv, page=page, weight=True, extra=sum(kept_pages) + 1, fill=0.0, seed=budget)
    bits = torch.uint8 if kv == "e4m3" else torch.int16
    for pool in (pc.k, pc.v):
        raw = pool.view(bits)
        raw.copy_(torch.randint(0, 100, raw.shape, generator=pc.gen, dtype=torch.int32).to(DEV).to(bits))
    w = torch.rand(pc.weight.shape, generator=pc.gen)
    if kind == "ties":
        w = (w ** 4 * 200).floor() / 8
    elif kind == "special":
        w = torch.where(w < 0.01, math.nan, torch.where(w < 0.02, math.inf, w))
    pc.weight.copy_(w.to(DEV))
    width = max(max(kept_pages), 1)
    dst = ints([[pc.free.pop() for _ in range(c)] + [-1] * (width - c) for c in kept_pages])
    before = [pc.k.clone(), pc.v.clone(), pc.weight.clone()]
    kept = torch.full((len(lens), heads, budget), 77, dtype=torch.int32, device=DEV)
    new = torch.full((len(lens),), 77, dtype=torch.int32, device=DEV)
    qg.check(qg.qg_kv_evict(pc.cache, pc.table, pc.width, dst, width, pc.lens, len(lens),
                            max(lens) if max_len is None else max_len, budget, sinks, recent, kept, new))
    torch.cuda.synchronize()
    assert qg.qg_device_status() == (0, 0)
    assert new.tolist() == [min(n, budget) for n in lens]
    for b, n in enumerate(lens):
        p, i = pc.where(b)
        want = definition(before[2][p, :, i].T.cpu(), n, budget, sinks, recent).to(DEV)
        m = want.shape[1]
        assert torch.equal(kept[b, :, :m].long(), want) and bool((kept[b, :, m:] == -1).all()), b
        to = torch.arange(m, device=DEV)
        for pool, old in zip((pc.k, pc.v, pc.weight), before):
            bit = bits if pool.dim() == 4 else torch.int32
            for h in range(heads):
                got = pool.view(bit)[dst[b].long()[to // page], h, to % page]
                src = old.view(bit)[pc.table[b].long()[want[h] // page], h, want[h] % page]
                assert torch.equal(got, src), (b, h)


@pytest.mark.parametrize("heads,n,budget,sinks", [(1, 5000, 512, 4), (1, 20000, 16384, 0), (4, 2048, 64, 64),
                                                  (8, 9001, 4096, 1), (30, 6000, 777, 100), (40, 33333, 1, 1)])
def test_windows_without_a_middle(qg, heads, n, budget, sinks):
    """sinks + recent == budget on clusters of two, four and eight blocks: no
    search precedes the blocks' exchange of counts."""
    for _ in range(3):
        run(qg, [n, 0, n // 2], heads, budget, sinks, budget - sinks)


@pytest.mark.parametrize("kind", ["ties", "distinct", "special"])
@pytest.mark.parametrize("n,budget,sinks,recent,page", [(50011, 20000, 4, 100, 16), (50011, 3, 1, 1, 7),
                                                        (70003, 65000, 0, 0, 64), (52000, 52000 - 1, 10, 3, 20)])
def test_more_slots_than_a_block_holds(qg, kind, n, budget, sinks, recent, page):
    """More heads than half the SMs: one block a head, over 1024 slots a warp
    and keys past the 49152 that shared memory holds."""
    run(qg, [n], 80, budget, sinks, recent, page=page, kind=kind)


def test_protected_ends_fill_the_budget_of_long_heads(qg):
    run(qg, [60001], 80, 50000, 20000, 30000)


def test_capacity_far_above_the_lengths(qg):
    """max_len is a capacity: blocks, threads and shared memory follow it."""
    for max_len in (1040, 5000 * 16, 200000 * 16):
        pc_lens = [1040, 300]
        kept = -(-600 // 16)
        pc = Paged(qg, pc_lens, 2, 16, "bf16", weight=True, extra=2 * kept + 1, fill=0.0, seed=3,
                   width=max(65, -(-max_len // 16))).fill()
        pc.weight.copy_(torch.rand(pc.weight.shape, generator=pc.gen).to(DEV))
        dst = ints([[pc.free.pop() for _ in range(kept)] for _ in range(2)])
        out = torch.empty(2, 2, 600, dtype=torch.int32, device=DEV)
        new = torch.empty(2, dtype=torch.int32, device=DEV)
        qg.check(qg.qg_kv_evict(pc.cache, pc.table, pc.width, dst, kept, pc.lens, 2, max_len, 600, 4, 40, out, new))
        torch.cuda.synchronize()
        assert qg.qg_device_status() == (0, 0) and new.tolist() == [600, 300]
        p, i = pc.where(0)
        assert torch.equal(out[0].long().cpu(), definition(pc.weight[p, :, i].T.cpu(), 1040, 600, 4, 40))
        assert out[1, :, :300].tolist() == [list(range(300))] * 2 and bool((out[1, :, 300:] == -1).all())


@pytest.mark.parametrize("budget", [2 ** 31 - 1, 2 ** 31 - 4000])
def test_budgets_up_to_the_largest_integer(qg, budget):
    """A budget that bounds nothing: all slots are kept, the rest of `kept` is -1."""
    pc = Paged(qg, [100], 1, 16, "bf16", weight=True, extra=8, fill=0.0, seed=5).fill()
    dst = ints([[pc.free.pop() for _ in range(7)]])
    kept = torch.full((budget + 8192,), 77, dtype=torch.int32, device=DEV)
    new = torch.empty(1, dtype=torch.int32, device=DEV)
    qg.check(qg.qg_kv_evict(pc.cache, pc.table, pc.width, dst, 7, pc.lens, 1, 100, budget, 4, 2000, kept, new))
    torch.cuda.synchronize()
    assert qg.qg_device_status() == (0, 0) and new.tolist() == [100]
    assert kept[:100].tolist() == list(range(100)) and bool((kept[100:budget] == -1).all())
    assert bool((kept[budget:] == 77).all())
