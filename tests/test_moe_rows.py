"""Rows to their experts and back on the GPU: dispatch (copied and as codes)
bit for bit, combine and its gradient against 64 bits, for every pair of
types, odd widths, strides, addresses, slots without a row, rows without a
slot, tokens without any row, infinities and NaN."""
import itertools

import pytest

torch = pytest.importorskip("torch")

from moe_util import (DEV, DTYPES, HALF, TINY, U, blocks, codes_of, guarded, ids_of, ints, routing,  # noqa: E402
                      sorted_slots, unharmed)

pytestmark = pytest.mark.gpu
WIDE = ("f32", "bf16", "f16")


@pytest.fixture(scope="module")
def qg():
    import weight_only_quantized_i4g_gb300 as m
    return m


def bits(t):
    return t.view({1: torch.uint8, 2: torch.int16, 4: torch.int32}[t.element_size()])


def randn(shape, dtype, seed, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * scale).to(DTYPES[dtype]).to(DEV)


def slots(tokens, k, experts=8, away=0.2, seed=0):
    _, order, place = sorted_slots(routing(tokens, k, experts, seed, away), experts)
    return place, len(order)


SIZES = [(1, 1, 1), (1, 8, 128), (3, 2, 7), (5, 3, 127), (2, 4, 129), (37, 6, 1999), (64, 1, 1024), (9, 8, 5120),
         (11, 3, 136), (4, 2, 2056), (2, 20, 72), (3, 2, 40000)]


@pytest.mark.parametrize("dtype", WIDE)
@pytest.mark.parametrize("tokens,k,width", SIZES)
def test_dispatch_copy(qg, dtype, tokens, k, width):
    place, n = slots(tokens, k)
    x = randn((tokens, width + 3), dtype, 1)[:, :width]              # an odd stride
    rows = guarded((n + 2, width), DTYPES[dtype])
    t = ids_of(qg)[dtype]
    qg.check(qg.qg_moe_dispatch(rows, t, None, x, t, width + 3, ints(place), tokens, k, width, n + 2))
    want = torch.full_like(rows, 7.0)
    for s, p in enumerate(place):
        if p >= 0:
            want[p] = x[s // k]
    assert torch.equal(bits(rows), bits(want)) and unharmed(rows)


@pytest.mark.parametrize("dtype", WIDE)
@pytest.mark.parametrize("tokens,k,width", SIZES)
@pytest.mark.parametrize("pad", [0, 5])
def test_dispatch_codes(qg, dtype, tokens, k, width, pad):
    place, n = slots(tokens, k)
    x = randn((tokens, width + pad), dtype, 2, 3.0)
    x[:, ::97] *= 50
    x[tokens // 2, : width // 2] *= 2.0 ** -14
    x = x[:, :width]
    rows, scale = guarded((n + 2, width), DTYPES["e4m3"]), guarded((n + 2, blocks(width)), torch.float32)
    qg.check(qg.qg_moe_dispatch(rows, qg.QG_E4M3, scale, x, ids_of(qg)[dtype], width + pad, ints(place), tokens, k,
                                width, n + 2))
    codes, s = codes_of(x)
    want = torch.full((n + 2, width), 0x38, dtype=torch.uint8)
    want_s = torch.full((n + 2, blocks(width)), 7.0)
    for slot, p in enumerate(place):
        if p >= 0:
            want[p] = codes.view(torch.uint8)[slot // k]
            want_s[p] = s[slot // k]
    assert torch.equal(scale.cpu(), want_s)
    assert torch.equal(rows.view(torch.uint8).cpu(), want)
    assert unharmed(rows) and unharmed(scale)


def test_codes_at_every_border(qg):
    """Block maxima around 448 * 2^e, values half-way between codes, subnormals, zeros, the types' ends."""
    v = []
    for e in (-126, -125, -100, -20, -9, -1, 0, 1, 7, 60, 119):
        for top in (448.0, 447.9999, 448.0001, 449.0, 256.0, 447.0, 255.9):
            block = [top * 2.0 ** e]
            block += [s * m * 2.0 ** (e - j) for j in range(0, 12) for m in (1.0, 1.0625, 1.1875, 1.9375, 1.5) for s in (1, -1)]
            v.append((block + [0.0, -0.0] + [0.0] * 128)[:128])
    v.append([0.0] * 128)
    v.append([2.0 ** -149] + [0.0] * 127)
    v.append([3.4e38, -3.4e38, 1.0] + [0.0] * 125)
    x = torch.tensor(v, dtype=torch.float64).clamp(-3.4e38, 3.4e38).float().to(DEV)
    n = x.shape[0]
    rows, scale = guarded((n, 128), DTYPES["e4m3"]), guarded((n, 1), torch.float32)
    qg.check(qg.qg_moe_dispatch(rows, qg.QG_E4M3, scale, x, qg.QG_F32, 128, None, n, 1, 128, n))
    codes, s = codes_of(x)
    assert torch.equal(scale.cpu(), s)
    assert torch.equal(rows.view(torch.uint8).cpu(), codes.view(torch.uint8))
    assert bool((s[-3] == 2.0 ** -126).all()) and bool((codes[-3].float() == 0).all())


@pytest.mark.parametrize("dtype", WIDE)
def test_codes_of_infinities_and_nan(qg, dtype):
    x = randn((3, 384), dtype, 4)
    x[0, 5], x[0, 200], x[1, 130] = float("inf"), float("nan"), float("-inf")
    x[2, 128:256] = float("nan")
    rows, scale = guarded((3, 384), DTYPES["e4m3"]), guarded((3, 3), torch.float32)
    qg.check(qg.qg_moe_dispatch(rows, qg.QG_E4M3, scale, x, ids_of(qg)[dtype], 384, None, 3, 1, 384, 3))
    codes, s = codes_of(x)
    assert torch.equal(scale.cpu(), s)
    got, want = rows.float().cpu(), codes.float()
    assert torch.equal(torch.isnan(got), torch.isnan(want)) and torch.equal(torch.isnan(got), ~torch.isfinite(x.float().cpu()))
    assert torch.equal(torch.nan_to_num(got), torch.nan_to_num(want))


def rows_of(y, place, tokens, k):
    """Each slot's row in 64 bits, zero for none: [tokens, k, width]."""
    p = torch.tensor(place, device=DEV)
    r = y[p.clamp_min(0)].double() if y.shape[0] else torch.zeros(len(place), y.shape[1], dtype=torch.float64, device=DEV)
    return torch.where((p < 0)[:, None], 0.0, r).view(tokens, k, -1)


def near(got, want, slack, dtype):
    err = (got.double() - want).abs()
    return bool((err <= slack + HALF[dtype] * (want.abs() + slack) + TINY[dtype]).all())


@pytest.mark.parametrize("yt,ot", list(itertools.product(WIDE, WIDE)))
@pytest.mark.parametrize("tokens,k,width", SIZES)
def test_combine(qg, yt, ot, tokens, k, width):
    place, n = slots(tokens, k)
    y, w = randn((n + 2, width), yt, 5), randn((tokens, k), "f32", 6)
    out = guarded((tokens, width), DTYPES[ot])
    t = ids_of(qg)
    qg.check(qg.qg_moe_combine(out, t[ot], y, t[yt], w, ints(place), tokens, k, width, n + 2))
    r = rows_of(y, place, tokens, k) * w.double()[..., None]
    # k fused steps, each off by half a step of a partial sum, which no sum of magnitudes is below
    assert near(out, r.sum(1), (k + 1) * U * r.abs().sum(1), ot) and unharmed(out)


@pytest.mark.parametrize("yt,ot", [("f32", "bf16"), ("bf16", "f32"), ("f16", "f16")])
@pytest.mark.parametrize("tokens,k,width", SIZES)
def test_combine_without_weights_or_places(qg, yt, ot, tokens, k, width):
    y = randn((tokens * k + 1, width), yt, 7)
    out = guarded((tokens, width), DTYPES[ot])
    t = ids_of(qg)
    qg.check(qg.qg_moe_combine(out, t[ot], y, t[yt], None, None, tokens, k, width, tokens * k + 1))
    r = rows_of(y, list(range(tokens * k)), tokens, k)
    assert near(out, r.sum(1), (k + 1) * U * r.abs().sum(1), ot) and unharmed(out)


def test_combine_reads_no_row_of_a_slot_without_one(qg):
    """Rows that no slot names hold NaN; places off the table's end count as none."""
    y = torch.full((6, 256), float("nan"), device=DEV)
    y[2] = 1.5
    w = torch.full((3, 2), float("inf"), device=DEV)
    w[0, 0] = 2.0
    place = ints([[2, -1], [6, -7], [2 ** 31 - 1, -2 ** 31]])
    out = guarded((3, 256), torch.bfloat16)
    qg.check(qg.qg_moe_combine(out, qg.QG_BF16, y, qg.QG_F32, w, place, 3, 2, 256, 6))
    assert bool((out[0] == 3.0).all()) and bool((out[1:] == 0).all())
    qg.check(qg.qg_moe_combine(out, qg.QG_BF16, None, qg.QG_F32, w, place, 3, 2, 256, 0))    # no rows at all
    assert bool((out == 0).all()) and unharmed(out)


@pytest.mark.parametrize("yt,dt", list(itertools.product(WIDE, WIDE)))
@pytest.mark.parametrize("tokens,k,width", SIZES)
def test_combine_grad(qg, yt, dt, tokens, k, width):
    place, n = slots(tokens, k, seed=2)
    y, w, d = randn((n + 2, width), yt, 8), randn((tokens, k), "f32", 9), randn((tokens, width), dt, 10)
    dy, dw = guarded((n + 2, width), DTYPES[yt]), guarded((tokens, k), torch.float32)
    t = ids_of(qg)
    qg.check(qg.qg_moe_combine_grad(dy, dw, d, t[dt], y, t[yt], w, ints(place), tokens, k, width, n + 2))
    want = torch.full((n + 2, width), 7.0, dtype=torch.float64, device=DEV)
    for s, p in enumerate(place):
        if p >= 0:
            want[p] = w.double().view(-1)[s] * d[s // k].double()
    assert near(dy, want, U * want.abs(), yt) and unharmed(dy)
    r = rows_of(y, place, tokens, k) * d.double()[:, None]
    # width terms in some order: each is rounded once on its way and takes part in at most width additions
    assert near(dw, r.sum(-1), (width + 1) * U * r.abs().sum(-1), "f32") and unharmed(dw)
    assert bool((dw.view(-1)[torch.tensor(place, device=DEV) < 0] == 0).all())


@pytest.mark.parametrize("what", ["dy", "dw"])
def test_combine_grad_half_wanted(qg, what):
    place, n = slots(50, 4, seed=3)
    y, w, d = randn((n, 520), "bf16", 8), randn((50, 4), "f32", 9), randn((50, 520), "bf16", 10)
    whole = [guarded((n, 520), torch.bfloat16), guarded((50, 4), torch.float32)]
    part = [guarded((n, 520), torch.bfloat16), guarded((50, 4), torch.float32)]
    a = (d, qg.QG_BF16, y, qg.QG_BF16, w, ints(place), 50, 4, 520, n)
    qg.check(qg.qg_moe_combine_grad(*whole, *a))
    if what == "dy":
        qg.check(qg.qg_moe_combine_grad(part[0], None, d, qg.QG_BF16, None, qg.QG_BF16, w, ints(place), 50, 4, 520, n))
        assert torch.equal(part[0], whole[0]) and bool((part[1] == 7).all())
    else:
        qg.check(qg.qg_moe_combine_grad(None, part[1], *a))
        assert torch.equal(part[1], whole[1]) and bool((part[0] == 7).all())


def test_gradients_against_differences(qg):
    """The scalar <dout, combine(y, w)> moves with y and w as the gradients say.  It is linear in each alone, so a
    difference over a whole step is exact up to the f32 sums of combine and gradient: (k + 1) and (width + 1)
    roundings of terms below, and 2^-24 of the outputs that the scalar multiplies."""
    tokens, k, width = 6, 3, 133
    place, n = slots(tokens, k, seed=5)
    y, w, d = randn((n, width), "f32", 8), randn((tokens, k), "f32", 9), randn((tokens, width), "f32", 10)
    pl = ints(place)

    def value(y, w):
        out = torch.empty(tokens, width, device=DEV)
        qg.check(qg.qg_moe_combine(out, qg.QG_F32, y, qg.QG_F32, w, pl, tokens, k, width, n))
        return (out.double() * d.double()).sum()
    dy, dw = torch.empty(n, width, device=DEV), torch.empty(tokens, k, device=DEV)
    qg.check(qg.qg_moe_combine_grad(dy, dw, d, qg.QG_F32, y, qg.QG_F32, w, pl, tokens, k, width, n))
    ty, tw = randn((n, width), "f32", 11), randn((tokens, k), "f32", 12)
    mag = 4 * (rows_of(y.abs() + ty.abs(), place, tokens, k) * (w.abs() + tw.abs()).double()[..., None] *
               d.abs().double()[:, None]).sum()
    y1, w1 = y + ty, w + tw
    got = value(y1, w) - value(y, w)
    assert abs(got - (dy.double() * (y1.double() - y.double())).sum()) <= (width + k + 4) * U * mag
    got = value(y, w1) - value(y, w)
    assert abs(got - (dw.double() * (w1.double() - w.double())).sum()) <= (width + k + 4) * U * mag


def test_dispatch_gradient_is_the_sum_of_its_rows(qg):
    """<combine(dispatch(x)) without weights>: dx = sum of the rows' gradients."""
    tokens, k, width = 40, 4, 264
    place, n = slots(tokens, k, seed=6)
    dr = randn((n, width), "bf16", 3)
    dx = guarded((tokens, width), torch.float32)
    qg.check(qg.qg_moe_combine(dx, qg.QG_F32, dr, qg.QG_BF16, None, ints(place), tokens, k, width, n))
    r = rows_of(dr, place, tokens, k)
    assert near(dx, r.sum(1), (k + 1) * U * r.abs().sum(1), "f32")


def test_far_rows(qg):
    """Rows beyond 2^31 bytes and elements."""
    width, n = 8192, 300000                                  # 2.4e9 codes
    rows = torch.zeros(n, width, dtype=torch.uint8, device=DEV)
    scale = torch.zeros(n, 64, device=DEV)
    x = randn((2, width), "bf16", 1)
    place = ints([[0, n - 1], [270001, -1]])
    qg.check(qg.qg_moe_dispatch(rows, qg.QG_E4M3, scale, x, qg.QG_BF16, width, place, 2, 2, width, n))
    codes, s = codes_of(x)
    for p, t in ((0, 0), (n - 1, 0), (270001, 1)):
        assert torch.equal(rows[p].cpu(), codes.view(torch.uint8)[t]) and torch.equal(scale[p].cpu(), s[t])
    assert int((rows != 0).sum(1).gt(0).sum()) == 3
    y = rows.view(torch.float16)                             # the same bytes as f16 rows of half the width
    out = torch.empty(2, width // 2, dtype=torch.float16, device=DEV)
    qg.check(qg.qg_moe_combine(out, qg.QG_F16, y, qg.QG_F16, None, ints([[n - 1], [270001]]), 2, 1, width // 2, n))
    ok = ~torch.isnan(y[n - 1])
    assert torch.equal(out[0][ok] + 0, y[n - 1][ok] + 0)
