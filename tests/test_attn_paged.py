"""Attention of new tokens over a paged cache on the GPU against its definition
in 64 bits: types, head layouts, lengths from none to long, page sizes that end
inside a tile, strides, drafted tokens, what masked slots hold, device-side
errors, streams, graphs and repeatability."""
import pytest

torch = pytest.importorskip("torch")

from attn_util import DEV, DTYPES, Paged, attention, check_attention, ids, ints, run_attention  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def qg():
    import weight_only_quantized_i4g_gb300 as m
    return m


def queries(pc, B, S, hq, kv, scale=1.5):
    return (scale * pc.randn(B * S, hq * pc.dim)).to(DTYPES["f16" if kv == "f16" else "bf16"])


RAGGED = [0, 1, 15, 16, 17, 31, 33, 64, 129, 300, 1000]


@pytest.mark.parametrize("kv", ["bf16", "f16", "e4m3"])
@pytest.mark.parametrize("dim", [16, 64, 80, 128, 160, 256])
def test_types_and_head_sizes(qg, kv, dim):
    pc = Paged(qg, RAGGED, 2, dim, kv, seed=dim).fill()
    q = queries(pc, len(RAGGED), 1, 6, kv)
    check_attention(pc, q, 1, 6, dim ** -0.5)


@pytest.mark.parametrize("kv", ["bf16", "f16", "e4m3"])
@pytest.mark.parametrize("out", ["f32", "bf16", "f16"])
def test_output_types(qg, kv, out):
    pc = Paged(qg, [70, 5, 260], 2, 128, kv, seed=3).fill()
    check_attention(pc, queries(pc, 3, 1, 10, kv), 1, 10, 0.09, out)


def test_e4m3_cache_with_f16_queries(qg):
    pc = Paged(qg, [70, 5, 260], 2, 128, "e4m3", seed=4).fill()
    q = (1.5 * pc.randn(3, 8 * 128)).half()
    check_attention(pc, q, 1, 8, 0.09)


@pytest.mark.parametrize("heads,group", [(1, 1), (1, 7), (8, 5), (3, 7), (2, 9), (1, 16), (2, 17), (1, 33), (1, 71)])
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_head_layouts(qg, heads, group, dim):
    pc = Paged(qg, [0, 3, 200, 47], heads, dim, "bf16", seed=group).fill()
    check_attention(pc, queries(pc, 4, 1, heads * group, "bf16"), 1, heads * group, dim ** -0.5)


@pytest.mark.parametrize("group", [9, 17, 33])
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("kv,out", [("bf16", "bf16"), ("f16", "f16"), ("e4m3", "bf16"), ("e4m3", "f32")])
def test_many_rows_by_output_type(qg, kv, out, dim, group):
    pc = Paged(qg, [0, 3, 200, 47], 2, dim, kv, seed=group).fill()
    check_attention(pc, queries(pc, 4, 1, 2 * group, kv), 1, 2 * group, dim ** -0.5, out)


@pytest.mark.parametrize("kv", ["bf16", "f16", "e4m3"])
@pytest.mark.parametrize("group,dim", [(8, 128), (16, 64), (32, 64), (32, 128)])
def test_long_sums_do_not_shrink(qg, kv, group, dim):
    """With positive V, sums rounded to nearest are off by a random walk, which
    the mean over all outputs leaves far below a unit.  What does not average
    out: a matrix instruction rounds towards zero, up to three a step of 16
    slots, each by 2^-23 of that step's own sum, and the parts of P leave 2^-22
    at most: 6e-7, taken as 1e-6.  Sums in the instruction's accumulators were
    2e-6 too small after 50 steps of a warp; here it has 60 and more."""
    B, n, heads = 48, 6000, 8
    pc = Paged(qg, [n], heads, dim, kv, seed=group)
    for h in range(heads):
        pc.put("k", 0, h, (20.0 if kv == "e4m3" else 1.0) * pc.randn(n, dim))
        pc.put("v", 0, h, (64.0 if kv == "e4m3" else 1.0) * (0.5 + torch.rand(n, dim, generator=pc.gen).to(DEV)))
    pc.table, pc.lens, pc.lens_list = pc.table.repeat(B, 1), ints([n] * B), [n] * B      # all read the same pages
    q = queries(pc, B, 1, heads * group, kv, 0.5)
    o, _ = run_attention(pc, q, 1, heads * group, dim ** -0.5)
    ref = attention(pc, q, 1, heads * group, dim ** -0.5)[0]
    bias = ((o.double().view_as(ref) - ref) / ref).mean().item()
    assert abs(bias) <= 1e-6, bias


@pytest.mark.parametrize("S", [1, 2, 3, 4, 5, 6, 7, 8])
@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
def test_drafted_tokens(qg, S, kv):
    """Sequences shorter than S have rows that see nothing."""
    lens = [0, 1, 2, 3, 7, 8, 9, 16, 17, 20, 24, 333]
    pc = Paged(qg, lens, 2, 128, kv, seed=S).fill()
    check_attention(pc, queries(pc, len(lens), S, 10, kv), S, 10, 0.088)


@pytest.mark.parametrize("page", [1, 3, 7, 16, 20, 24, 32, 64, 100, 128, 256])
def test_page_sizes(qg, page):
    pc = Paged(qg, [1, 40, 130, 257], 2, 128, "bf16", page=page, seed=page).fill()
    check_attention(pc, queries(pc, 4, 1, 8, "bf16"), 1, 8, 0.088)


@pytest.mark.parametrize("order", ["head", "token"])
@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
def test_page_orders(qg, order, kv):
    pc = Paged(qg, [37, 150], 4, 128, kv, order=order, seed=9).fill()
    check_attention(pc, queries(pc, 2, 2, 8, kv), 2, 8, 0.088)


def test_interleaved_pools_and_strided_queries(qg):
    """k and v of a page side by side in one allocation; q a slice of wider rows."""
    base = Paged(qg, [37, 150, 90], 4, 64, "bf16", seed=10)
    both = torch.full((base.n_pages, 2, 4, 16, 64), float("nan"), dtype=torch.bfloat16, device=DEV)
    base.k, base.v = both[:, 0], both[:, 1]
    base.cache = qg.kv_cache(base.k, base.v)
    base.fill()
    wide = (1.5 * base.randn(3, 8 * 64 + 96)).bfloat16()
    q = wide[:, 32:32 + 8 * 64]
    o64 = attention(base, q, 1, 8, 0.125)[0]
    o = torch.empty(3, 8, 64, device=DEV)
    n = qg.qattn_workspace_bytes(base.cache, 3, 150, 1, 8)
    ws = torch.empty(max(n, 1), dtype=torch.uint8, device=DEV)
    qg.check(qg.qattn_paged(base.cache, base.table, base.width, base.lens, 3, 150, o, qg.QG_F32, None, q, qg.QG_BF16,
                            wide.shape[1], 1, 8, 0.125, 0, ws, n))
    assert float((o.double() - o64[:, 0]).abs().max()) < 2e-4        # |v| <= 5, bf16 inputs exact


@pytest.mark.parametrize("kv,n", [("bf16", 40000), ("e4m3", 70001)])
def test_long_sequences(qg, kv, n):
    pc = Paged(qg, [n, 0, 17, n // 3], 1, 128, kv, page=64, seed=11).fill()
    check_attention(pc, queries(pc, 4, 1, 5, kv), 1, 5, 0.088, accumulate=False)


@pytest.mark.parametrize("B", [1, 3, 200, 1500])
def test_batch_sizes(qg, B):
    """From one sequence to more than a block has threads; ages unequal."""
    lens = [(i * 37) % 61 for i in range(B)]
    lens[0] = 900
    pc = Paged(qg, lens, 1, 64, "bf16", seed=B).fill()
    check_attention(pc, queries(pc, B, 1, 3, "bf16"), 1, 3, 0.125)


@pytest.mark.parametrize("kv", ["bf16", "f16", "e4m3"])
@pytest.mark.parametrize("S,group", [(1, 1), (1, 5), (3, 4), (8, 7)])
def test_weights_are_accumulated(qg, kv, S, group):
    lens = [0, 1, 2, 18, 250, 1031]
    pc = Paged(qg, lens, 2, 128, kv, seed=S + group, weight=True).fill()
    q = queries(pc, len(lens), S, 2 * group, kv)
    check_attention(pc, q, S, 2 * group, 0.088, accumulate=True)
    check_attention(pc, q, S, 2 * group, 0.088, accumulate=True, lse=False)


@pytest.mark.parametrize("dim,S,group", [(64, 8, 7), (64, 8, 9), (128, 4, 6), (128, 8, 9), (256, 2, 5), (256, 8, 5)])
def test_weights_of_many_rows(qg, dim, S, group):
    """Rows that several warps, or several segments, share out."""
    lens = [0, 5, 77, 700]
    pc = Paged(qg, lens, 2, dim, "bf16", seed=dim + S, weight=True).fill()
    q = queries(pc, len(lens), S, 2 * group, "bf16")
    check_attention(pc, q, S, 2 * group, dim ** -0.5, accumulate=True)


@pytest.mark.parametrize("accumulate", [False, True])
def test_more_sequences_than_a_launch_takes(qg, accumulate):
    """Their lengths sit in shared memory, 2048 at a time."""
    B = 4100
    lens = [(i * 7) % 23 for i in range(B)]
    lens[2047], lens[2048], lens[4099] = 300, 290, 280
    pc = Paged(qg, lens, 1, 16, "bf16", page=16, seed=41, weight=accumulate, fill=0.0)
    n = sum(lens)
    for name in ("k", "v"):                       # one write for all sequences
        at = torch.cat([torch.arange(x) for x in lens]).to(DEV)
        seq = torch.repeat_interleave(torch.arange(B), torch.tensor(lens)).to(DEV)
        getattr(pc, name)[pc.table[seq, at // 16].long(), 0, at % 16] = pc.randn(n, 16).bfloat16()
    q = queries(pc, B, 1, 2, "bf16")
    o, lse = run_attention(pc, q, 1, 2, 0.25, accumulate=accumulate)
    torch.cuda.synchronize()
    assert qg.qg_device_status() == (0, 0)
    for b in (0, 1, 22, 23, 2046, 2047, 2048, 2049, 3000, 4098, 4099):
        if lens[b] == 0:
            assert bool((o[b] == 0).all())
            continue
        k, v = pc.get("k", b, 0), pc.get("v", b, 0)
        z = q[b].double().view(2, 16) @ k.T * 0.25
        p = torch.softmax(z, -1)
        assert float((o[b].double() - p @ v).abs().max()) < 1e-4
        assert float((lse[b].double() - torch.logsumexp(z, -1)).abs().max()) < 1e-4
        if accumulate:
            at, i = pc.where(b)
            assert float((pc.weight[at, 0, i].double() - 0.25 - p.sum(0)).abs().max()) < 1e-4


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("kv", ["bf16", "f16", "e4m3"])
@pytest.mark.parametrize("S", [2, 4, 8])
def test_masked_slots_never_touch_their_rows(qg, bad, kv, S):
    """The newest slot is hidden from every row but the last: those rows stay
    what they are without it, whatever k and v hold there."""
    if kv == "e4m3" and bad != bad:
        pass
    elif kv == "e4m3":
        pytest.skip("e4m3 has no infinity")
    lens = [20, 33, 130]
    pc = Paged(qg, lens, 1, 128, kv, seed=S, fill=0.0).fill()
    q = queries(pc, 3, S, 6, kv)
    ref = attention(pc, q, S, 6, 0.088)[0]
    for b, n in enumerate(lens):
        for name in ("k", "v"):
            x = pc.get(name, b, 0)
            if kv == "e4m3":
                x = x / getattr(pc, name + "_scale")[0].double()
            x[n - 1] = bad
            pc.put(name, b, 0, x.float())
    o, _ = run_attention(pc, q, S, 6, 0.088)
    o = o.double().view(3, S, 6, 128)
    assert bool(torch.isfinite(o[:, :S - 1]).all())
    assert float((o[:, :S - 1] - ref[:, :S - 1]).abs().max()) < 1e-3 * float(ref.abs().max())
    if bad != bad:
        assert bool(torch.isnan(o[:, S - 1]).all())


def test_large_and_equal_scores(qg):
    """Scores of a few hundred and rows of equal scores: the maximum is taken out first."""
    pc = Paged(qg, [200, 45], 1, 128, "bf16", seed=21).fill()
    q = queries(pc, 2, 1, 4, "bf16", scale=20.0)
    q[:, :128] = 0
    check_attention(pc, q, 1, 4, 1.0)
    check_attention(pc, q, 1, 4, -1.0)
    check_attention(pc, q, 1, 4, 0.0)


def test_lowest_and_infinite_scores(qg):
    """A slot whose score is -inf weighs nothing beside finite ones; rows of
    only such slots are empty."""
    pc = Paged(qg, [40, 3], 1, 64, "bf16", seed=22).fill()
    x = pc.get("k", 0, 0)
    x[7] = 0
    x[7, 0] = -float("inf")
    pc.put("k", 0, 0, x.float())
    y = torch.zeros(3, 64, device=DEV)
    y[:, 0] = -float("inf")
    pc.put("k", 1, 0, y)
    q = torch.zeros(2, 64, device=DEV, dtype=torch.bfloat16)
    q[:, 0] = 1.0
    o, lse = run_attention(pc, q, 1, 1, 1.0)
    keep = [t for t in range(40) if t != 7]
    z = x[keep, 0]
    ref = (torch.softmax(z, 0)[:, None] * pc.get("v", 0, 0)[keep]).sum(0)
    assert float((o[0, 0].double() - ref).abs().max()) < 1e-4
    assert bool((o[1] == 0).all()) and float(lse[1, 0]) == -float("inf")


def test_pages_outside_the_pool(qg):
    """Their rows are NaN, the others stand, the error word says so once."""
    pc = Paged(qg, [40, 50], 1, 64, "bf16", seed=23, weight=True).fill()
    q = queries(pc, 2, 1, 2, "bf16")
    ref = attention(pc, q, 1, 2, 0.1)[0]
    for bad in (pc.n_pages, -1, 2 ** 30, -2 ** 31):
        good = pc.table.clone()
        pc.table[1, 1] = bad
        o, lse = run_attention(pc, q, 1, 2, 0.1, accumulate=True)
        torch.cuda.synchronize()
        assert qg.qg_device_status() == (0, qg.QG_EPAGE)
        assert qg.qg_device_status() == (0, 0)
        assert float((o[0].double() - ref[0, 0]).abs().max()) < 1e-4
        assert bool(torch.isnan(o[1]).all()) and bool(torch.isnan(lse[1]).all())
        pc.table.copy_(good)


def test_lengths_outside_are_held(qg):
    pc = Paged(qg, [40, 48], 1, 64, "bf16", seed=24).fill()
    q = queries(pc, 2, 1, 2, "bf16")
    ref = attention(pc, q, 1, 2, 0.1)[0]
    pc.lens.copy_(ints([-5, 1 << 30]))
    o, lse = run_attention(pc, q, 1, 2, 0.1, max_len=48)
    torch.cuda.synchronize()
    assert qg.qg_device_status() == (0, qg.QG_EPAGE)
    assert bool((o[0] == 0).all()) and float((o[1].double() - ref[1, 0]).abs().max()) < 1e-4


def test_offsets_past_32_bits(qg):
    """A pool of more than 4 GiB whose used pages lie at its far end."""
    heads, dim, page = 1, 128, 16
    pages = (5 << 30) // (heads * dim * page * 2)
    k = torch.zeros(pages, heads, page, dim, dtype=torch.bfloat16, device=DEV)
    v = torch.zeros_like(k)
    small = Paged(qg, [100], heads, dim, "bf16", seed=25).fill()
    far = small.table + (pages - small.n_pages)
    k[pages - small.n_pages:] = small.k
    v[pages - small.n_pages:] = small.v
    q = queries(small, 1, 1, 4, "bf16")
    near, lse = run_attention(small, q, 1, 4, 0.1)
    small.cache, small.table = qg.kv_cache(k, v), far
    o, lse2 = run_attention(small, q, 1, 4, 0.1)
    assert torch.equal(o, near) and torch.equal(lse, lse2)


@pytest.mark.parametrize("accumulate", [False, True])
def test_repeats_are_identical_and_streams_are_used(qg, accumulate):
    lens = [3000, 10, 700, 1500]
    pc = Paged(qg, lens, 2, 128, "bf16", seed=26, weight=accumulate).fill()
    q = queries(pc, 4, 1, 8, "bf16")
    o, lse = run_attention(pc, q, 1, 8, 0.088, accumulate=accumulate)
    w = pc.weight.clone() if accumulate else None
    side = torch.cuda.Stream()
    for _ in range(3):
        if accumulate:
            pc.weight.fill_(0.25)
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            o2, lse2 = run_attention(pc, q, 1, 8, 0.088, accumulate=accumulate)
        side.synchronize()
        assert torch.equal(o, o2) and torch.equal(lse, lse2)
        if accumulate:
            assert torch.equal(w, pc.weight)


def test_graph_replays_with_new_lengths(qg):
    pc = Paged(qg, [400, 30], 2, 128, "bf16", seed=27).fill()
    q = queries(pc, 2, 1, 8, "bf16")
    o = torch.empty(2, 8, 128, device=DEV)
    n = qg.qattn_workspace_bytes(pc.cache, 2, 400, 1, 8)
    ws = torch.empty(max(n, 1), dtype=torch.uint8, device=DEV)

    def call():
        qg.check(qg.qattn_paged(pc.cache, pc.table, pc.width, pc.lens, 2, 400, o, qg.QG_F32, None, q, qg.QG_BF16,
                                8 * 128, 1, 8, 0.088, 0, ws, n))
    call()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    for lens in ([400, 30], [17, 30], [0, 29], [399, 1]):
        pc.lens.copy_(ints(lens))
        pc.lens_list = lens
        g.replay()
        torch.cuda.synchronize()
        ref = attention(pc, q, 1, 8, 0.088)[0]
        assert float((o.double() - ref[:, 0]).abs().max()) < 1e-4


def test_no_sequences(qg):
    pc = Paged(qg, [5], 1, 64, "bf16").fill()
    n0 = qg.qg_launch_count()
    assert qg.qattn_paged(pc.cache, pc.table, 1, pc.lens, 0, 5, pc.k, 0, None, pc.k, 1, 64, 1, 1, 0.1) == qg.QG_OK
    assert qg.qg_launch_count() == n0
    assert ids(qg)["bf16"] == 1
