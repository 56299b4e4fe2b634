"""Rotary positions and the cache write on the GPU against the definition in 64
bits: input, query and cache types, both pair orders, partial rotation, several
axes, far positions, padding tokens, strides, saturation and NaN, and places
that are not in the cache."""
import math

import pytest

torch = pytest.importorskip("torch")

from attn_util import DEV, DTYPES, HALF_ULP, Paged, ids, ints  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def qg():
    import weight_only_quantized_i4g_gb300 as m
    return m


def definition(x, pos, axis, freq, rotary, interleaved):
    """x f64 [T, heads, dim] turned."""
    out = x.clone()
    for j in range(rotary // 2):
        i0, i1 = (2 * j, 2 * j + 1) if interleaved else (j, j + rotary // 2)
        a = pos[:, axis[j]].double() * freq[j].double()
        c, s = a.cos()[:, None], a.sin()[:, None]
        out[..., i0] = x[..., i0] * c - x[..., i1] * s
        out[..., i1] = x[..., i1] * c + x[..., i0] * s
    return out


def near(got, want, dtype, mag):
    """One rounding to the type over an f32 rotation (a few 2^-24 of |x| + |y|,
    the sine and cosine within 2^-22)."""
    return bool(((got.double() - want).abs() <= HALF_ULP[dtype] * want.abs() + 2.0 ** -20 * mag + 2.0 ** -25).all())


def call(qg, pc, seq, slot, q, qkv, src, hq, pos, axis, freq, rotary, interleaved, qt, T=None, stride=None):
    return qg.qg_rope_append(pc.cache, pc.table, pc.width, len(pc.lens_list), seq, slot,
                             seq.numel() if T is None else T, q, ids(qg)[qt], qkv, ids(qg)[src],
                             stride or qkv.stride(0), hq, pos, pos.shape[1], axis, freq, rotary,
                             qg.QG_ROPE_INTERLEAVED if interleaved else qg.QG_ROPE_HALF)


CASES = [  # src, kv, q type, T, hq, hkv, dim, rotary, axes, interleaved, page, order
    ("f32", "bf16", "bf16", 1, 5, 1, 128, 128, 1, False, 16, "head"),
    ("f32", "f16", "f16", 7, 8, 8, 64, 64, 1, True, 16, "head"),
    ("f32", "e4m3", "bf16", 9, 14, 2, 128, 64, 1, False, 64, "head"),
    ("bf16", "bf16", "bf16", 33, 6, 2, 80, 40, 2, False, 24, "head"),
    ("f16", "bf16", "f16", 5, 6, 2, 80, 40, 2, True, 7, "token"),
    ("bf16", "e4m3", "f16", 200, 4, 1, 256, 256, 3, True, 16, "token"),
    ("f32", "bf16", "bf16", 50, 3, 3, 16, 6, 3, False, 1, "head"),
    ("f32", "bf16", "bf16", 50, 3, 3, 24, 22, 3, True, 5, "head"),
    ("f32", "e4m3", "bf16", 12, 2, 1, 32, 0, 1, False, 16, "head"),
    ("f32", "e4m3", "f16", 700, 56, 8, 128, 128, 3, False, 64, "head"),
]


@pytest.mark.parametrize("src,kv,qt,T,hq,hkv,dim,rotary,axes,interleaved,page,order", CASES)
def test_against_the_definition(qg, src, kv, qt, T, hq, hkv, dim, rotary, axes, interleaved, page, order):
    n_seq = min(3, T)
    per = [T // n_seq + (b < T % n_seq) for b in range(n_seq)]
    past = [5 * b for b in range(n_seq)]
    pc = Paged(qg, [a + b for a, b in zip(per, past)], hkv, dim, kv, page=page, order=order, weight=True, fill=0.0,
               seed=T)
    seq = ints([b for b in range(n_seq) for _ in range(per[b])])
    slot = ints([past[b] + i for b in range(n_seq) for i in range(per[b])])
    shuffle = torch.randperm(T, generator=pc.gen).to(DEV)      # tokens in any order
    seq, slot = seq[shuffle].contiguous(), slot[shuffle].contiguous()
    pos = torch.randint(0, 30000, (T, axes), generator=pc.gen, dtype=torch.int32).to(DEV)
    axis = bytes((3 * j) % axes for j in range(rotary // 2))
    freq = (10000.0 ** (-torch.arange(rotary // 2, dtype=torch.float64) * 2 / max(rotary, 1))).float().to(DEV)
    row = (hq + 2 * hkv) * dim
    wide = pc.randn(T, row + 8).to(DTYPES[src])
    qkv = wide[:, :row]
    q = torch.full((T, hq * dim), float("nan"), dtype=DTYPES[qt], device=DEV)
    k0, v0 = pc.k.clone(), pc.v.clone()
    qg.check(call(qg, pc, seq, slot, q, qkv, src, hq, pos, axis, freq, rotary, interleaved, qt))
    torch.cuda.synchronize()
    assert qg.qg_device_status() == (0, 0)
    x = qkv.double().reshape(T, hq + 2 * hkv, dim)
    turned = definition(x[:, :hq + hkv], pos, axis, freq, rotary, interleaved)
    mag = 5.0 + x.abs().max()
    assert near(q.view(T, hq, dim), turned[:, :hq], qt, mag)
    written = torch.zeros(pc.n_pages, page, dtype=torch.bool, device=DEV)
    p = pc.table[seq.long(), slot.long() // page].long()
    i = slot.long() % page
    written[p, i] = True
    assert int(written.sum()) == T
    for pool, before, want, scale in ((pc.k, k0, turned[:, hq:], pc.k_scale), (pc.v, v0, x[:, hq + hkv:], pc.v_scale)):
        bits = torch.uint8 if kv == "e4m3" else torch.int16
        raw, old = pool.view(bits), before.view(bits)
        if order == "token":
            raw, old = raw.transpose(1, 2), old.transpose(1, 2)
        got = raw[p, :, i].view(pool.dtype).double()
        if kv == "e4m3":
            y = want / scale.double()[:, None]
            # half an ulp of a 4-bit significand, subnormals in steps of 2^-9
            assert bool(((got - y.clamp(-448, 448)).abs() <= 2.0 ** -4 * y.abs() * 1.001 + 2.0 ** -10 * 1.001).all())
        else:
            assert near(got, want, kv, mag)
        keep = ~written[:, None, :, None].expand(raw.shape)
        assert torch.equal(raw[keep], old[keep])               # nothing else was touched
    w = torch.where(written[:, None, :], 0.0, 0.25).expand_as(pc.weight)
    assert torch.equal(pc.weight, w)


def test_far_positions(qg):
    """Positions up to 2^31 - 1: the angle is reduced in 64 bits."""
    T, dim = 16, 128
    pc = Paged(qg, [T], 1, dim, "f16", fill=0.0)
    pos = ints([0, 1, 2, 1000, 65535, 1 << 20, 12345678, 1 << 24, (1 << 24) + 1, 1 << 28, 987654321, 2 ** 31 - 1,
                2 ** 30, -1, -1000, 3]).view(T, 1)
    freq = (10000.0 ** (-torch.arange(64, dtype=torch.float64) / 64)).float().to(DEV)
    qkv = pc.randn(T, 3 * dim)
    q = torch.empty(T, dim, dtype=torch.float16, device=DEV)
    qg.check(call(qg, pc, ints([0] * T), ints(list(range(T))), q, qkv, "f32", 1, pos, None, freq, dim, False, "f16"))
    want = definition(qkv.double().view(T, 3, dim)[:, :2], pos, [0] * 64, freq, dim, False)
    assert near(q.view(T, 1, dim), want[:, :1], "f16", 5 + float(qkv.abs().max()))


def test_padding_and_missing_places(qg):
    T, dim = 6, 64
    pc = Paged(qg, [20, 5], 2, dim, "bf16", fill=0.0, weight=True)
    qkv = pc.randn(T, 6 * dim)
    q = torch.full((T, 2 * dim), float("nan"), dtype=torch.bfloat16, device=DEV)
    pos, freq = torch.zeros(T, 1, dtype=torch.int32, device=DEV), torch.ones(32, device=DEV)
    qg.check(call(qg, pc, ints([0] * T), ints([-1] * T), q, qkv, "f32", 2, pos, None, freq, dim, False, "bf16"))
    torch.cuda.synchronize()
    assert qg.qg_device_status() == (0, 0)
    # position 0 and frequencies of one: no turn
    assert torch.equal(q, qkv[:, :2 * dim].bfloat16()) and not bool(pc.k.any()) and not bool(pc.v.any())
    # a sequence, a slot past the table, a table entry that names no page
    for seq, slot in ((2, 0), (-1, 0), (0, pc.width * 16), (1, 16), (0, 2 ** 31 - 1)):
        qg.check(call(qg, pc, ints([seq]), ints([slot]), q, qkv, "f32", 2, pos, None, freq, dim, False, "bf16", T=1))
        torch.cuda.synchronize()
        assert qg.qg_device_status() == (0, qg.QG_EPAGE), (seq, slot)
        assert not bool(pc.k.any()) and not bool(pc.v.any()) and bool((pc.weight == 0.25).all())
    n0 = qg.qg_launch_count()
    assert call(qg, pc, ints([0]), ints([0]), q, qkv, "f32", 2, pos, None, freq, dim, False, "bf16", T=0) == qg.QG_OK
    assert qg.qg_launch_count() == n0


def test_e4m3_saturates_and_keeps_nan(qg):
    dim = 32
    pc = Paged(qg, [1], 1, dim, "e4m3", fill=0.0)
    row = torch.zeros(1, 3 * dim, device=DEV)
    row[0, dim:dim + 5] = torch.tensor([1e30, -1e30, math.inf, -math.inf, math.nan], device=DEV)
    row[0, 2 * dim:2 * dim + 3] = torch.tensor([math.nan, 1e30, 0.0], device=DEV)
    q = torch.empty(1, dim, dtype=torch.bfloat16, device=DEV)
    qg.check(call(qg, pc, ints([0]), ints([0]), q, row, "f32", 1, ints([[0]]), None,
                  torch.ones(1, device=DEV), 0, False, "bf16"))
    p, i = pc.where(0)
    k = pc.k.view(torch.uint8)[p, 0, i].view(torch.float8_e4m3fn)[0].float().tolist()
    v = pc.v.view(torch.uint8)[p, 0, i].view(torch.float8_e4m3fn)[0].float().tolist()
    assert k[:4] == [448.0, -448.0, 448.0, -448.0] and math.isnan(k[4])
    assert math.isnan(v[0]) and v[1:3] == [448.0, 0.0]
