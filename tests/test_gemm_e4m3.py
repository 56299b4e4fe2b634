"""Products of e4m3 activations and weights on the GPU against 64 bits: one
row to many, widths that end inside a block, empty and ragged experts, rows
outside every expert, both scale encodings, every output type, NaN codes, every
alignment, offsets that lead out of the rows."""
import pytest

torch = pytest.importorskip("torch")

from moe_util import DEV, DTYPES, HALF, TINY, blocks, guarded, ids_of, ints, product, unharmed  # noqa: E402

pytestmark = pytest.mark.gpu
E4M3 = torch.float8_e4m3fn


@pytest.fixture(scope="module")
def qg():
    import weight_only_quantized_i4g_gb300 as m
    return m


def codes(shape, seed, spread=100.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * spread).clamp(-448, 448).to(E4M3).to(DEV)


def scales(shape, seed, power):
    g = torch.Generator().manual_seed(seed)
    if power:
        return torch.randint(110, 120, shape, generator=g, dtype=torch.uint8).to(DEV)
    return torch.exp(torch.rand(shape, generator=g) * 4.6 - 9.2).to(DEV)


def as_f32(ws):
    return torch.exp2(ws.double() - 127).float() if ws.dtype == torch.uint8 else ws


def call(qg, y, x, xs, w, ws, offsets=None, yt=None, stream=None):
    m, (e, o, i) = x.shape[0], w.shape
    fmt = qg.QG_FMT_FP8UE8M0 if ws.dtype == torch.uint8 else qg.QG_FMT_FP8B128
    t = ids_of(qg)[yt or {v: k for k, v in DTYPES.items()}[y.dtype]]
    wb = qg.qgemm_e4m3_workspace_bytes(m, i, o, e)
    wk = torch.full((max(wb, 1),), 0xFF, dtype=torch.uint8, device=DEV)
    if offsets is None:
        return qg.qgemm_e4m3(fmt, y, t, x, xs, w, ws, m, i, o, wk, wb, stream)
    return qg.qgemm_e4m3_moe(fmt, y, t, x, xs, w, ws, offsets, e, m, i, o, wk, wb, stream)


def held(y, want, mag, yt):
    """The documented bound (1e-3 of the magnitudes summed), and the output's rounding."""
    err = (y.double() - want).abs()
    return bool((err <= 1e-3 * mag * (1 + HALF[yt]) + HALF[yt] * want.abs() + TINY[yt]).all())


DENSE = [(1, 16, 1), (1, 128, 128), (1, 7168, 256), (3, 272, 130), (8, 2048, 500), (17, 1040, 129), (33, 128, 1000),
         (64, 4096, 128), (65, 512, 384), (130, 640, 200), (200, 1152, 1), (257, 256, 257), (300, 2064, 640), (700, 384, 513),
         (1024, 1024, 1024), (16, 16384, 128), (513, 5120, 264), (3001, 1040, 1500), (2500, 128, 2100), (129, 16384, 2050)]


@pytest.mark.parametrize("m,i,o", DENSE)
@pytest.mark.parametrize("power", [False, True])
@pytest.mark.parametrize("yt", ["f32", "bf16", "f16"])
def test_dense(qg, m, i, o, power, yt):
    x, w = codes((m, i), 1, 20.0), codes((1, o, i), 2, 20.0)
    xs, ws = scales((m, blocks(i)), 3, False), scales((1, blocks(o), blocks(i)), 4, power)
    y = guarded((m, o), DTYPES[yt])
    qg.check(call(qg, y, x, xs, w, ws))
    want, mag = product(x, xs, w, as_f32(ws), [0, m])
    assert held(y, want, mag, yt) and unharmed(y)


@pytest.mark.parametrize("m,i,o", [(5, 1, 3), (7, 100, 129), (66, 131, 70), (40, 1999, 65)])
def test_widths_of_no_whole_lines(qg, m, i, o):
    x, w = codes((m, i), 1), codes((1, o, i), 2)
    xs, ws = scales((m, blocks(i)), 3, False), scales((1, blocks(o), blocks(i)), 4, False)
    y = guarded((m, o), torch.float32)
    qg.check(call(qg, y, x, xs, w, ws))
    want, mag = product(x, xs, w, ws, [0, m])
    assert held(y, want, mag, "f32") and unharmed(y)


@pytest.mark.parametrize("ax,aw,ay", [(1, 0, 0), (0, 8, 0), (0, 0, 2), (4, 4, 2)])
def test_odd_addresses(qg, ax, aw, ay):
    m, i, o = 50, 272, 140
    x, w = codes((m, i), 1), codes((1, o, i), 2)
    xs, ws = scales((m, blocks(i)), 3, False), scales((1, blocks(o), blocks(i)), 4, False)
    xo = torch.zeros(m * i + 64, dtype=torch.uint8, device=DEV)
    wo = torch.zeros(o * i + 64, dtype=torch.uint8, device=DEV)
    yo = torch.zeros(m * o * 2 + 64, dtype=torch.uint8, device=DEV)
    x2 = xo[ax:ax + m * i].view(E4M3).view(m, i)
    w2 = wo[aw:aw + o * i].view(E4M3).view(1, o, i)
    x2.view(torch.uint8).copy_(x.view(torch.uint8))
    w2.view(torch.uint8).copy_(w.view(torch.uint8))
    y = yo[ay:ay + 2 * m * o].view(torch.bfloat16).view(m, o)
    qg.check(call(qg, y, x2, xs, w2, ws))
    want, mag = product(x, xs, w, ws, [0, m])
    assert held(y, want, mag, "bf16")


GROUPS = [([1], 128, 128), ([0, 1, 0], 256, 130), ([1] * 8, 7168, 256), ([0, 0, 5], 272, 128), ([3, 0, 17, 64, 0, 1], 512, 200),
          ([64, 64, 64, 64], 256, 128), ([100, 1, 0, 300, 28], 640, 264), ([0] * 30 + [7] + [0] * 33, 384, 150),
          ([13] * 37, 256, 384), ([700, 2, 65], 384, 513), ([2, 1] * 40, 1152, 128), ([255, 257, 256, 1], 1024, 300),
          ([900, 0, 129, 1, 1000, 128, 640], 1040, 1380), ([300] * 9 + [0] * 700 + [17] * 300, 128, 400)]


@pytest.mark.parametrize("counts,i,o", GROUPS)
@pytest.mark.parametrize("power,yt", [(False, "f32"), (True, "bf16"), (False, "f16")])
def test_grouped(qg, counts, i, o, power, yt):
    e, n = len(counts), sum(counts)
    bounds = [0]
    for c in counts:
        bounds.append(bounds[-1] + c)
    m = n + 3                                                 # rows behind the last expert's stay as they were
    x, w = codes((m, i), 1, 20.0), codes((e, o, i), 2, 20.0)
    xs, ws = scales((m, blocks(i)), 3, False), scales((e, blocks(o), blocks(i)), 4, power)
    y = guarded((m, o), DTYPES[yt])
    qg.check(call(qg, y, x, xs, w, ws, ints(bounds)))
    want, mag = product(x, xs, w, as_f32(ws), bounds)
    assert held(y[:n], want[:n], mag[:n], yt)
    assert bool((y[n:] == 7).all()) and unharmed(y)
    assert qg.qg_device_status() == (qg.QG_OK, qg.QG_OK)


@pytest.mark.parametrize("m,i,o", [(1, 256, 128), (8, 4096, 384), (70, 1024, 130), (300, 2048, 512), (1100, 512, 256)])
def test_small_integers_are_exact(qg, m, i, o):
    """Codes of small integers and scales of powers of two: every partial sum is a whole number of 2^-8 below 2^24 such
    units, so any order of f32 sums gives the definition itself."""
    g = torch.Generator().manual_seed(5)
    x = torch.randint(-4, 5, (m, i), generator=g).float().to(E4M3).to(DEV)
    w = torch.randint(-4, 5, (1, o, i), generator=g).float().to(E4M3).to(DEV)
    xs = torch.exp2(torch.randint(-4, 0, (m, blocks(i)), generator=g).float()).to(DEV)
    ws = torch.randint(123, 127, (1, blocks(o), blocks(i)), generator=g, dtype=torch.uint8).to(DEV)
    y = guarded((m, o), torch.float32)
    qg.check(call(qg, y, x, xs, w, ws))
    want, mag = product(x, xs, w, as_f32(ws), [0, m])
    assert float(mag.max()) < 2.0 ** 16
    assert torch.equal(y.double(), want)


def test_every_code(qg):
    """One element of a row at a time: Y[m, o] is a product of two codes and two scales, for all 256 x 256."""
    i = 256
    x = torch.zeros(256, i, dtype=torch.uint8, device=DEV)
    x[:, 37] = torch.arange(256, dtype=torch.uint8, device=DEV)
    w = torch.zeros(1, 256, i, dtype=torch.uint8, device=DEV)
    w[0, :, 37] = torch.arange(256, dtype=torch.uint8, device=DEV)
    x, w = x.view(E4M3), w.view(E4M3)
    xs, ws = torch.full((256, 2), 0.5, device=DEV), torch.full((1, 2, 2), 0.25, device=DEV)
    y = guarded((256, 256), torch.float32)
    qg.check(call(qg, y, x, xs, w, ws))
    want, _ = product(x, xs, w, ws, [0, 256])
    assert torch.equal(torch.isnan(y), torch.isnan(want))
    assert torch.equal(torch.nan_to_num(y.double()), torch.nan_to_num(want))


def test_nan_stays_in_its_row_and_column(qg):
    counts, bounds = [20, 40], [0, 20, 60]
    x, w = codes((64, 512), 1), codes((2, 300, 512), 2)
    x.view(torch.uint8)[30, 300] = 0x7F
    w.view(torch.uint8)[0, 170, 9] = 0xFF
    x.view(torch.uint8)[61, 3] = 0x7F                         # behind the last expert's rows: in nobody's way
    xs, ws = scales((64, 4), 3, False), scales((2, 3, 4), 4, False)
    y = guarded((64, 300), torch.float32)
    qg.check(call(qg, y, x, xs, w, ws, ints(bounds)))
    nan = torch.zeros(64, 300, dtype=torch.bool, device=DEV)
    nan[30] = True
    nan[:20, 170] = True
    assert sum(counts) == 60 and torch.equal(torch.isnan(y), nan)
    assert bool((y[60:] == 7).all())


@pytest.mark.parametrize("counts,i,o", [([3, 0, 30], 272, 130), ([900, 700, 1], 1040, 1300), ([3, 30], 271, 70)])
def test_rows_before_the_first_expert_stay(qg, counts, i, o):
    bounds = [11]
    for c in counts:
        bounds.append(bounds[-1] + c)
    m = bounds[-1] + 2
    x, w = codes((m, i), 1), codes((len(counts), o, i), 2)
    xs, ws = scales((m, blocks(i)), 3, False), scales((len(counts), blocks(o), blocks(i)), 4, False)
    y = guarded((m, o), torch.bfloat16)
    qg.check(call(qg, y, x, xs, w, ws, ints(bounds)))
    want, mag = product(x, xs, w, ws, bounds)
    assert held(y[11:-2], want[11:-2], mag[11:-2], "bf16")
    assert bool((y[:11] == 7).all()) and bool((y[-2:] == 7).all()) and unharmed(y)


@pytest.mark.parametrize("scale", [2.0 ** -40, 2.0 ** 40, 0.0])
def test_scales_far_from_one(qg, scale):
    """Scales whose product is a normal f32 keep every bit: times a power of two the result is the same bits, scaled."""
    m, i, o = 70, 640, 140
    x, w = codes((m, i), 1), codes((1, o, i), 2)
    xs, ws = scales((m, 5), 3, False), scales((1, 2, 5), 4, False)
    y, z = guarded((m, o), torch.float32), guarded((m, o), torch.float32)
    qg.check(call(qg, y, x, xs, w, ws))
    qg.check(call(qg, z, x, xs * scale, w, ws))
    assert torch.equal(z, y * scale)


@pytest.mark.parametrize("m,o", [(20, 200), (1500, 1300)])
def test_infinite_and_nan_scales_stay_in_their_tokens(qg, m, o):
    x, w = codes((m, 384), 1), codes((1, o, 384), 2)
    xs, ws = scales((m, 3), 3, False), scales((1, blocks(o), 3), 4, False)
    xs[5, 1], xs[7, 2] = float("inf"), float("nan")
    y = guarded((m, o), torch.float32)
    qg.check(call(qg, y, x, xs, w, ws))
    bad = ~torch.isfinite(y)
    assert bool(bad[5].all()) and bool(bad[7].all()) and int(bad.any(1).sum()) == 2


@pytest.mark.parametrize("table", [[0, 10, 5, 30], [-5, 10, 20, 30], [0, 10, 20, 99], [40, 50, 2 ** 31 - 1, -2 ** 31]])
def test_offsets_that_lead_out_of_the_rows(qg, table):
    m, i, o = 40, 256, 128
    x, w = codes((m, i), 1), codes((3, o, i), 2)
    xs, ws = scales((m, 2), 3, False), scales((3, 1, 2), 4, False)
    y = guarded((m, o), torch.float32)
    qg.check(call(qg, y, x, xs, w, ws, ints(table)))
    assert qg.qg_device_status() == (qg.QG_OK, qg.QG_EEXPERT)
    assert qg.qg_device_status() == (qg.QG_OK, qg.QG_OK)
    assert unharmed(y)
    if table == [-5, 10, 20, 30]:                              # the good rows are right all the same
        want, mag = product(x, xs, w, ws, [0, 10, 20, 30])
        assert held(y[:30], want[:30], mag[:30], "f32") and bool((y[30:] == 7).all())


def test_repeats_and_other_streams_give_the_same_bits(qg):
    counts = [31, 0, 140, 8, 1]
    bounds = [0, 31, 31, 171, 179, 180]
    assert sum(counts) == 180
    x, w = codes((180, 4096), 1), codes((5, 384, 4096), 2)
    xs, ws = scales((180, 32), 3, False), scales((5, 3, 32), 4, False)
    off = ints(bounds)
    first = torch.empty(180, 384, device=DEV)
    qg.check(call(qg, first, x, xs, w, ws, off))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = []
    for n in range(6):                                         # two streams at once, a workspace each
        with torch.cuda.stream(streams[n % 2]):
            y = torch.empty(180, 384, device=DEV)
            qg.check(call(qg, y, x, xs, w, ws, off))
            outs.append(y)
    torch.cuda.synchronize()
    assert all(torch.equal(first, y) for y in outs)
