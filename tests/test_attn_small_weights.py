"""Attention where one slot draws nearly all weight and holds a zero v, so that
the output is made of the light slots: their weights must keep their bits.

Scores here are exact up to their last steps (q has one element, a power of
two): a score in log2 units, up to 40, is a product and a difference rounded in
f32 with a factor rounded twice, within 4 * 2^-24 * 40 of the true one, which
moves its power of two by 7e-6 relatively; 2^x itself is within 2^-22.  P keeps
16 bits down to 2^-32 of the heaviest weight (2^-16), products and sums in f32
add less than 2^-19.  So 2^-15 of sum p |v| bounds the error up to 22 nats."""
import math

import pytest

torch = pytest.importorskip("torch")

from attn_util import DEV, DTYPES, Paged, attention, run_attention  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def qg():
    import weight_only_quantized_i4g_gb300 as m
    return m


def check(qg, kv, gap, at, out="f32", lens=(2000, 300), heads=1, group=4, dim=128, S=1, spread=0.03, max_len=None):
    pc = Paged(qg, lens, heads, dim, kv, seed=int(gap) + dim)
    unit = 256.0 if kv == "e4m3" else 8.0           # the heavy slot's first element
    if kv == "e4m3":
        pc.k_scale.fill_(2.0 ** -6)
        pc.v_scale.fill_(2.0 ** -5)
    for b, n in enumerate(lens):
        heavy = int(at * (n - S))
        for h in range(heads):
            k = (20.0 if kv == "e4m3" else 1.0) * pc.randn(n, dim)
            k[:, 0] = unit * spread * torch.randn(n, generator=pc.gen).to(DEV)
            k[heavy, 0] = unit
            v = (100.0 if kv == "e4m3" else 1.0) * (0.5 + torch.rand(n, dim, generator=pc.gen).to(DEV))
            v[heavy] = 0.0
            pc.put("k", b, h, k)
            pc.put("v", b, h, v)
    q = torch.zeros(len(lens) * S, heads * group, dim, device=DEV)
    q[..., 0] = 2.0 ** -(torch.arange(heads * group, device=DEV) % 2)      # every other row has half the gap
    q = q.view(len(lens) * S, -1).to(DTYPES["f16" if kv == "f16" else "bf16"])
    scale = gap / (unit * (2.0 ** -6 if kv == "e4m3" else 1.0))
    ref, lse, _, mag, _ = attention(pc, q, S, heads * group, scale)
    o, l = run_attention(pc, q, S, heads * group, scale, out, max_len=max_len)
    torch.cuda.synchronize()
    assert qg.qg_device_status() == (0, 0)
    half = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8, "f16": 2.0 ** -11}[out]
    err = (o.double().view_as(ref) - ref).abs()
    bound = 2.0 ** -15 * mag + half * ref.abs() + (2.0 ** -25 if out == "f16" else 0.0)
    assert bool((err <= bound).all()), float((err / mag).max())
    assert float((l.double().view_as(lse) - lse).abs().max()) < 1e-5
    assert not math.isnan(float(o.float().sum()))


@pytest.mark.parametrize("kv", ["bf16", "f16", "e4m3"])
@pytest.mark.parametrize("at", [0.0, 0.003, 0.5, 1.0])
@pytest.mark.parametrize("gap", [8, 12, 16, 20, 22])
def test_light_slots_beside_a_heavy_one(qg, kv, at, gap):
    check(qg, kv, gap, at)


@pytest.mark.parametrize("kv,out", [("bf16", "bf16"), ("f16", "f16"), ("f16", "f32"), ("e4m3", "bf16"), ("e4m3", "f32")])
@pytest.mark.parametrize("group,dim,S", [(1, 64, 1), (12, 64, 1), (8, 64, 8), (12, 128, 1), (24, 128, 1), (8, 128, 8),
                                         (4, 256, 1), (12, 256, 1), (8, 256, 4)])
def test_light_slots_in_every_kernel(qg, kv, out, group, dim, S):
    check(qg, kv, 20, 0.1, out, (900, 33), 1, group, dim, S)


@pytest.mark.parametrize("kv", ["f16", "e4m3"])
def test_light_slots_of_equal_scores(qg, kv):
    """Their errors do not average out."""
    check(qg, kv, 20, 0.0, spread=0.0)


@pytest.mark.parametrize("kv", ["f16", "e4m3"])
def test_light_slots_over_many_blocks(qg, kv):
    """Equal ranges of all steps, joined by the second kernel."""
    check(qg, kv, 20, 0.7, lens=(40000, 500, 7000), heads=2)
