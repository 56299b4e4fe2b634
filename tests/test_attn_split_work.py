"""Attention where all steps are cut into equal ranges over the SMs, segments
span blocks and a second kernel joins them: element by element against the
definition, over types, row counts, new tokens and weights.

More segments than SMs, or more K and V in a sequence than eight blocks take
whole, lead there; each case below is one of the two."""
import pytest

torch = pytest.importorskip("torch")

from attn_util import DEV, Paged, attention, check_attention, run_attention  # noqa: E402
from test_attn_paged import queries  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def qg():
    import weight_only_quantized_i4g_gb300 as m
    return m


MANY = [0, 1, 15, 16, 17, 31, 64, 129, 300, 5, 77, 200] * 7          # 84 sequences of two cache heads: 168 segments


def tall(kv, dim, heads):
    """Lengths of a few sequences, the longest above eight blocks' 384 KB."""
    n = 8 * (384 << 10) // (dim * 2 * (1 if kv == "e4m3" else 2)) + 37
    return [n, 3, 0, n // 5 + 1, 700][:5 if heads == 1 else 3]


# cache heads, rows a cache head = S * group: one to four row tiles a warp, groups of warps, several segments a head
KINDS = [("bf16", "bf16", True), ("bf16", "f32", False), ("f16", "f16", True), ("e4m3", "bf16", False), ("e4m3", "f32", True)]
ROWS = [(1, 1), (1, 5), (4, 2), (1, 12), (4, 4), (3, 7), (4, 8), (8, 6), (8, 8), (8, 10)]


@pytest.mark.parametrize("kv,out,accumulate", KINDS)
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("S,group", ROWS)
def test_many_segments(qg, kv, out, dim, S, group, accumulate):
    pc = Paged(qg, MANY, 2, dim, kv, seed=dim + S + group, weight=accumulate).fill()
    check_attention(pc, queries(pc, len(MANY), S, 2 * group, kv), S, 2 * group, dim ** -0.5, out, accumulate)


@pytest.mark.parametrize("kv,out,accumulate", KINDS)
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("S,group", ROWS)
def test_long_segments(qg, kv, out, dim, S, group, accumulate):
    lens = tall(kv, dim, 1)
    pc = Paged(qg, lens, 1, dim, kv, page=64, seed=dim + S + group, weight=accumulate).fill()
    check_attention(pc, queries(pc, len(lens), S, group, kv), S, group, dim ** -0.5, out, accumulate)


@pytest.mark.parametrize("page,order", [(1, "head"), (7, "token"), (24, "head"), (100, "token")])
@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
def test_pages_that_end_inside_a_step(qg, kv, page, order):
    pc = Paged(qg, MANY, 2, 128, kv, page=page, order=order, seed=page, weight=True).fill()
    check_attention(pc, queries(pc, len(MANY), 3, 10, kv), 3, 10, 0.088, "f32", True)


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("kv", ["bf16", "f16", "e4m3"])
@pytest.mark.parametrize("S,group", [(2, 3), (4, 4), (8, 8)])
def test_hidden_slots_never_touch_their_rows(qg, bad, kv, S, group):
    if kv == "e4m3" and bad == bad:
        bad = float("nan")                            # e4m3 has no infinity
    lens = tall(kv, 128, 1)
    pc = Paged(qg, lens, 1, 128, kv, page=16, seed=S, fill=0.0).fill()
    q = queries(pc, len(lens), S, group, kv)
    ref, _, _, mag, _ = attention(pc, q, S, group, 0.088)
    for b, n in enumerate(lens):
        for name in ("k", "v"):
            if n:
                x = pc.get(name, b, 0)
                if kv == "e4m3":
                    x = x / getattr(pc, name + "_scale")[0].double()
                x[n - 1] = bad
                pc.put(name, b, 0, x.float())
    o, _ = run_attention(pc, q, S, group, 0.088)
    o = o.double().view(len(lens), S, group, 128)
    assert bool(torch.isfinite(o[:, :S - 1]).all())
    assert bool(((o - ref)[:, :S - 1].abs() <= 1e-3 * mag[:, :S - 1]).all())
    if bad != bad:
        assert bool(torch.isnan(o[:, S - 1][torch.tensor([n > 0 for n in lens])]).all())


@pytest.mark.parametrize("kv", ["bf16", "f16", "e4m3"])
@pytest.mark.parametrize("S,group", [(1, 5), (4, 8), (8, 8)])
def test_repeats_are_identical(qg, kv, S, group):
    for lens, heads in ((MANY, 2), (tall(kv, 128, 1), 1)):
        pc = Paged(qg, lens, heads, 128, kv, seed=S, weight=True).fill()
        q = queries(pc, len(lens), S, heads * group, kv)
        first = None
        for _ in range(4):
            pc.weight.fill_(0.25)
            got = (*run_attention(pc, q, S, heads * group, 0.088, accumulate=True), pc.weight.clone())
            first = first or got
            assert all(torch.equal(a, b) for a, b in zip(first, got))


@pytest.mark.parametrize("kv", ["bf16", "f16", "e4m3"])
@pytest.mark.parametrize("group,dim,out", [(8, 128, "f32"), (16, 64, "bf16"), (32, 64, "bf16"), (32, 128, "bf16"),
                                           (32, 128, "f32"), (16, 128, "bf16"), (12, 256, "bf16")])
def test_long_sums_element_by_element(qg, kv, group, dim, out):
    """60 steps and more a warp, positive V.  check_attention's bound, and what it
    does not know: sums in the instructions' accumulators (bf16 output of more
    than 8 rows) lose 2^-24.4 a step and up to 2^-23 a part, 60 to 200 steps: a
    mean of up to 2e-5 below the definition's, far under a unit of bf16.  A mean
    over bf16 outputs is taken against the definition rounded alike: outputs
    crowd around 1, where rounding by itself has a mean."""
    B, n, heads = 20, 6000, 8
    pc = Paged(qg, [n], heads, dim, kv, seed=group)
    for h in range(heads):
        pc.put("k", 0, h, (20.0 if kv == "e4m3" else 1.0) * pc.randn(n, dim))
        pc.put("v", 0, h, (64.0 if kv == "e4m3" else 1.0) * (0.5 + torch.rand(n, dim, generator=pc.gen).to(DEV)))
    pc.table, pc.lens, pc.lens_list = pc.table.repeat(B, 1), pc.lens.repeat(B), [n] * B
    q = queries(pc, B, 1, heads * group, kv, 0.5)
    ref = attention(pc, q, 1, heads * group, dim ** -0.5)[0]
    o, _ = check_attention(pc, q, 1, heads * group, dim ** -0.5, out)
    mean = ((o.double().view_as(ref) - (ref if out == "f32" else ref.bfloat16().double())) / ref).mean().item()
    assert abs(mean) <= (2e-5 + 1e-5 if out == "bf16" else 1e-6), mean
