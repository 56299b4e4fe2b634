"""Sums of the e4m3 products beyond the documented bound: whole numbers that
f32 holds and 16 bits do not, exactly, in every kernel, output type and scale
encoding; general codes and scales within what f32 sums allow; and the
products of a backward pass through frozen weights."""
import pytest

torch = pytest.importorskip("torch")

from moe_util import DEV, DTYPES, HALF, TINY, U, blocks, guarded, ints, product, unharmed  # noqa: E402
from test_gemm_e4m3 import E4M3, as_f32, call, codes, qg, scales  # noqa: E402, F401

pytestmark = pytest.mark.gpu

# one matrix: few tokens (32, 64 and 128 a tile, K split or not), many tokens, the general kernel (2047: no whole lines)
DENSE = [(1, 16384, 128), (8, 7168, 300), (33, 4096, 130), (64, 16384, 256), (100, 2048, 2000), (128, 7168, 640), (300, 16384, 264),
         (700, 5120, 1300), (2100, 1152, 2050), (40, 2047, 70)]
GROUPS = [([1] * 8, 7168, 256), ([3, 0, 17, 64, 0, 1], 2048, 200), ([100, 1, 0, 300, 28], 4096, 264), ([700, 2, 65, 1000], 5120, 1300),
          ([3, 0, 17], 2047, 70)]


def whole(shape, seed):
    """Whole numbers 4 .. 12, one in eight negative: a block's sum is mostly above 2048, where f16 and bf16 have gaps."""
    g = torch.Generator().manual_seed(seed)
    v = torch.randint(4, 13, shape, generator=g)
    return torch.where(torch.rand(shape, generator=g) < 0.125, -v, v).float().to(E4M3).to(DEV)


def bounds_of(counts):
    out = [0]
    for c in counts:
        out.append(out[-1] + c)
    return out


@pytest.mark.parametrize("power,yt", [(False, "f32"), (True, "f32"), (False, "bf16"), (True, "f16")])
@pytest.mark.parametrize("counts,i,o", [([m], i, o) for m, i, o in DENSE] + GROUPS)
def test_whole_numbers_are_exact(qg, counts, i, o, power, yt):  # noqa: F811
    """|x w| <= 144 and scales of 1/2 or 1 on either side: every partial sum is a whole number of quarters, at most
    4 * 144 * 16384 < 2^24 of them, so f32 holds it whatever the order, and the output is the definition rounded once.
    (Outputs of 16 bits have scales 2^-8 below: the largest is then below f16's 65504.)"""
    e, bounds = len(counts), bounds_of(counts)
    m = bounds[-1]
    x, w = whole((m, i), 1), whole((e, o, i), 2)
    g = torch.Generator().manual_seed(3)
    down = 0 if yt == "f32" else 8
    xs = torch.exp2(torch.randint(-1 - down, 1 - down, (m, blocks(i)), generator=g).float()).to(DEV)
    ws = torch.randint(126, 128, (e, blocks(o), blocks(i)), generator=g, dtype=torch.uint8).to(DEV)
    if not power:
        ws = as_f32(ws)
    y = guarded((m, o), DTYPES[yt])
    qg.check(call(qg, y, x, xs, w, ws, ints(bounds) if e > 1 else None))
    want, mag = product(x, xs, w, as_f32(ws), bounds)
    assert float(mag.max()) * 2.0 ** (2 + down) < 2.0 ** 24
    assert torch.equal(y, want.to(DTYPES[yt])) and unharmed(y)


@pytest.mark.parametrize("power", [False, True])
@pytest.mark.parametrize("counts,i,o", [([m], i, o) for m, i, o in DENSE] + GROUPS)
def test_general_sums_stay_within_f32(qg, counts, i, o, power):  # noqa: F811
    """In units of U = 2^-24 of the magnitudes: a block's 128 exact products in any order of f32 additions, each off by
    less than a step (2 U, as a sum cut off rather than rounded is), 256; the product of the scales 1; a block's
    multiplication and addition 1 for each of the blocks; up to 8 partial sums of a split K, 8."""
    e, bounds = len(counts), bounds_of(counts)
    m = bounds[-1]
    x, w = codes((m, i), 1, 60.0), codes((e, o, i), 2, 60.0)
    xs, ws = scales((m, blocks(i)), 3, False), scales((e, blocks(o), blocks(i)), 4, power)
    y = guarded((m, o), torch.float32)
    qg.check(call(qg, y, x, xs, w, ws, ints(bounds) if e > 1 else None))
    want, mag = product(x, xs, w, as_f32(ws), bounds)
    assert bool(((y.double() - want).abs() <= (265 + blocks(i)) * U * mag).all()) and unharmed(y)


@pytest.mark.parametrize("m,i,o,power", [(5, 384, 256, False), (70, 272, 640, True), (600, 1040, 400, False)])
def test_backward_of_the_activations(qg, m, i, o, power):  # noqa: F811
    """dX = dY W for frozen weights: the same call on the codes and scales transposed (128 x 128 blocks become such
    blocks), dY as codes by qg_moe_dispatch; against 64 bits on those codes, with the bound above."""
    w, ws = codes((1, o, i), 2, 60.0), scales((1, blocks(o), blocks(i)), 4, power)
    dy = torch.randn(m, o, generator=torch.Generator().manual_seed(5)).bfloat16().to(DEV)
    c, s = torch.empty(m, o, dtype=E4M3, device=DEV), torch.empty(m, blocks(o), device=DEV)
    qg.check(qg.qg_moe_dispatch(c, qg.QG_E4M3, s, dy, qg.QG_BF16, o, None, m, 1, o, m))
    wt = w[0].view(torch.uint8).t().contiguous().view(E4M3)[None]
    dx = guarded((m, i), torch.bfloat16)
    qg.check(call(qg, dx, c, s, wt, ws[0].t().contiguous()[None]))
    full = as_f32(ws)[0].double().repeat_interleave(128, 0)[:o].repeat_interleave(128, 1)[:, :i] * w[0].double()
    grad = c.double() * s.double().repeat_interleave(128, 1)[:, :o]
    want, slack = grad @ full, (265 + blocks(o)) * U * (grad.abs() @ full.abs())
    err = (dx.double() - want).abs()
    assert bool((err <= slack + HALF["bf16"] * (want.abs() + slack) + TINY["bf16"]).all()) and unharmed(dx)
