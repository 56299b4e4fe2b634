"""Eviction by accumulated attention weight on the GPU against a plain sort:
which slots are kept (exactly), what is copied (bit for bit), ties, protected
ends, budgets of one and of everything, special weights, long sequences, page
sizes and orders, missing pages."""
import math

import pytest

torch = pytest.importorskip("torch")

from attn_util import DEV, Paged, ints  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def qg():
    import weight_only_quantized_i4g_gb300 as m
    return m


def setup(qg, lens, heads, dim, kv, page, budget, order="head", seed=0):
    """A filled cache with room for the survivors, and the table of that room."""
    kept = [min(n, budget) for n in lens]
    need = [-(-n // page) for n in kept]
    pc = Paged(qg, lens, heads, dim, kv, page=page, order=order, weight=True, extra=sum(need) + 1, fill=0.0, seed=seed)
    pc.fill()
    width = max(max(need), -(-min(budget, max(lens)) // page), 1)
    dst = [[-1] * width for _ in lens]
    for b, n in enumerate(need):
        for i in range(n):
            dst[b][i] = pc.free.pop()
    return pc, ints(dst), width


def definition(w, n, budget, sinks, recent):
    """Kept slots of one head, by a stable sort (largest first, NaN above all, -0 = 0)."""
    if n <= budget:
        return list(range(n))
    mid = [t for t in range(n) if sinks <= t < n - recent]
    rank = lambda t: (math.inf, 1) if math.isnan(w[t]) else (w[t] + 0.0, 0)  # noqa: E731
    best = sorted(mid, key=lambda t: (-rank(t)[0], -rank(t)[1], t))[:budget - sinks - recent]
    return sorted(set(range(sinks)) | set(range(n - recent, n)) | set(best))


def rows(pc, pool, table, b, h, slots):
    """Bits of the given slots of one head."""
    t = torch.tensor(slots, device=DEV, dtype=torch.long)
    p, i = table[b].long()[t // pc.page], t % pc.page
    raw = pool.view(torch.uint8) if pool.dtype == torch.float8_e4m3fn else pool.view(torch.int16) \
        if pool.dim() == 4 else pool.view(torch.int32)
    return raw[p, h, i] if pc.order == "head" or pool.dim() == 3 else raw[p, i, h]


def evict(qg, pc, dst, width, budget, sinks, recent, max_len=None):
    B = len(pc.lens_list)
    kept = torch.full((B, pc.heads, budget), 77, dtype=torch.int32, device=DEV)
    new = torch.full((B,), 77, dtype=torch.int32, device=DEV)
    qg.check(qg.qg_kv_evict(pc.cache, pc.table, pc.width, dst, width, pc.lens, B,
                            max(pc.lens_list) if max_len is None else max_len, budget, sinks, recent, kept, new))
    torch.cuda.synchronize()
    return kept, new


def check(qg, pc, dst, width, budget, sinks, recent):
    src = [pc.k.clone(), pc.v.clone(), pc.weight.clone()]
    want = {}
    for b, n in enumerate(pc.lens_list):
        for h in range(pc.heads):
            p, i = pc.where(b)
            want[b, h] = definition(pc.weight[p, h, i].tolist(), n, budget, sinks, recent)
    kept, new = evict(qg, pc, dst, width, budget, sinks, recent)
    assert qg.qg_device_status() == (0, 0)
    assert new.tolist() == [min(n, budget) for n in pc.lens_list]
    written = torch.zeros(pc.n_pages, pc.heads, pc.page, dtype=torch.bool, device=DEV)
    for (b, h), slots in want.items():
        assert kept[b, h].tolist() == slots + [-1] * (budget - len(slots)), (b, h)
        if not slots:
            continue
        for pool, old in zip((pc.k, pc.v, pc.weight), src):
            got = rows(pc, pool, dst, b, h, list(range(len(slots))))
            assert torch.equal(got, rows(pc, old, pc.table, b, h, slots)), (b, h)
        t = torch.arange(len(slots), device=DEV)
        written[dst[b].long()[t // pc.page], h, t % pc.page] = True
    for pool, old in zip((pc.k, pc.v), src):                      # nothing else was touched
        keep = ~(written if pc.order == "head" else written.transpose(1, 2))
        bits = torch.uint8 if pool.dtype == torch.float8_e4m3fn else torch.int16
        assert torch.equal(pool.view(bits)[keep], old.view(bits)[keep])
    assert torch.equal(pc.weight.view(torch.int32)[~written], src[2].view(torch.int32)[~written])   # NaN too


@pytest.mark.parametrize("kv,dim,page,order", [("bf16", 128, 16, "head"), ("f16", 64, 7, "head"),
                                               ("e4m3", 16, 24, "token"), ("e4m3", 256, 64, "head"),
                                               ("bf16", 80, 1, "token")])
@pytest.mark.parametrize("budget,sinks,recent", [(1, 0, 0), (1, 1, 0), (1, 0, 1), (40, 4, 8), (100, 0, 0),
                                                 (100, 60, 40), (333, 3, 30)])
def test_layouts_and_budgets(qg, kv, dim, page, order, budget, sinks, recent):
    lens = [0, 1, 39, 40, 41, 100, 101, 334, 700]
    pc, dst, width = setup(qg, lens, 2, dim, kv, page, budget, order, seed=budget)
    pc.weight.copy_(torch.rand(pc.weight.shape, generator=pc.gen).to(DEV))
    check(qg, pc, dst, width, budget, sinks, recent)


@pytest.mark.parametrize("kind", ["equal", "few", "zero signs", "special", "wide"])
@pytest.mark.parametrize("budget", [17, 256, 1000])
def test_weights(qg, kind, budget):
    lens = [1200, 300, 2500]
    pc, dst, width = setup(qg, lens, 2, 16, "bf16", 16, budget, seed=budget)
    w = torch.rand(pc.weight.shape, generator=pc.gen)
    if kind == "equal":
        w.fill_(0.5)
    elif kind == "few":
        w = (w * 4).floor()
    elif kind == "zero signs":
        w = torch.where(w < 0.5, -0.0, 0.0) + torch.where(w > 0.95, w, torch.tensor(-0.0))
    elif kind == "special":
        w = torch.where(w < 0.1, math.nan, torch.where(w < 0.2, math.inf, torch.where(w < 0.3, -math.inf, w - 0.6)))
    else:
        w = torch.exp(60 * (w - 0.5))
    pc.weight.copy_(w.to(DEV))
    check(qg, pc, dst, width, budget, 4, 10)


@pytest.mark.parametrize("n,budget,page", [(60000, 20000, 64), (130001, 4096, 100), (70000, 69999, 16)])
def test_long_sequences(qg, n, budget, page):
    pc, dst, width = setup(qg, [n, 33], 1, 16, "e4m3", page, budget, seed=n)
    pc.weight.copy_((torch.rand(pc.weight.shape, generator=pc.gen) ** 8 * 1000).floor().to(DEV) / 8)
    check(qg, pc, dst, width, budget, 4, 100)


def test_missing_pages(qg):
    """A source page outside the pool: its slots rank last and are not copied."""
    pc, dst, width = setup(qg, [64], 1, 16, "bf16", 16, 48)
    pc.weight.copy_(torch.rand(pc.weight.shape, generator=pc.gen).to(DEV) + 0.5)
    pc.table[0, 1] = pc.n_pages + 3
    k0 = pc.k.clone()
    kept, new = evict(qg, pc, dst, width, 48, 0, 0)
    assert kept[0, 0].tolist() == [t for t in range(64) if not 16 <= t < 32] and new.tolist() == [48]
    assert qg.qg_device_status() == (0, 0)
    kept, new = evict(qg, pc, dst, width, 48, 20, 0)              # slots 16 .. 19 are protected
    assert qg.qg_device_status() == (0, qg.QG_EPAGE)
    # a destination page outside the pool is not written
    pc.table[0, 1] = pc.table[0, 0]
    pc.k.copy_(k0)
    dst.fill_(-7)
    evict(qg, pc, dst, width, 48, 0, 0)
    assert qg.qg_device_status() == (0, qg.QG_EPAGE)
    assert torch.equal(pc.k, k0)


def test_lengths_outside_are_held(qg):
    pc, dst, width = setup(qg, [64, 40], 1, 16, "bf16", 16, 32)
    pc.lens.copy_(ints([1 << 30, -3]))
    kept, new = evict(qg, pc, dst, width, 32, 0, 32, max_len=64)
    assert qg.qg_device_status() == (0, qg.QG_EPAGE)
    assert new.tolist() == [32, 0] and kept[0, 0].tolist() == list(range(32, 64)) and int(kept[1].max()) == -1


def test_repeats_are_identical(qg):
    pc, dst, width = setup(qg, [5000, 900], 4, 64, "bf16", 16, 700)
    pc.weight.copy_((torch.rand(pc.weight.shape, generator=pc.gen) * 50).floor().to(DEV))
    a = evict(qg, pc, dst, width, 700, 4, 64)
    k = pc.k.clone()
    for _ in range(3):
        b = evict(qg, pc, dst, width, 700, 4, 64)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1]) and torch.equal(k, pc.k)
