"""Infinities in slots that rows do see: o is the sum of exp(z - lse) v, so an
element is infinite where v is (of one sign), NaN where both signs or a NaN
meet, and all other elements are what they are without it."""
import pytest

torch = pytest.importorskip("torch")

from attn_util import HALF_ULP, Paged, attention, run_attention  # noqa: E402
from test_attn_paged import queries  # noqa: E402

pytestmark = pytest.mark.gpu
INF = float("inf")


@pytest.fixture(scope="module")
def qg():
    import weight_only_quantized_i4g_gb300 as m
    return m


def check(qg, kv, out, lens, heads, group, dim, S, page=16, max_len=None):
    pc = Paged(qg, lens, heads, dim, kv, page=page, seed=dim + group).fill()
    for b, n in enumerate(lens):
        for h in range(heads):
            if n == 0:
                continue
            v = pc.get("v", b, h).float()
            v[n // 2, 1] = INF                       # one of each sign, in elements of their own
            v[n // 3, 6] = -INF
            v[0, 3], v[n - 1, 3] = INF, -INF         # the last new token sees both
            v[n - 1, dim - 2] = float("nan")
            v[: (n + 1) // 2, dim - 1] = INF         # many of one sign
            pc.put("v", b, h, v)
    q = queries(pc, len(lens), S, heads * group, kv)
    ref = attention(pc, q, S, heads * group, dim ** -0.5)[0]
    o, _ = run_attention(pc, q, S, heads * group, dim ** -0.5, out, max_len=max_len)
    torch.cuda.synchronize()
    assert qg.qg_device_status() == (0, 0)
    o = o.double().view_as(ref)
    assert torch.equal(o.isnan(), ref.isnan())
    assert torch.equal(o.isinf(), ref.isinf()) and torch.equal(o[o.isinf()], ref[ref.isinf()])
    fine = torch.isfinite(ref)
    assert bool(((o - ref).abs() <= HALF_ULP[out] * ref.abs() + 1e-3)[fine].all())      # |v| <= 5, scores within 1e-4
    assert bool(ref.isinf().any()) and bool(ref.isnan().any())


@pytest.mark.parametrize("kv,out", [("bf16", "bf16"), ("bf16", "f32"), ("f16", "f16"), ("f16", "f32")])
@pytest.mark.parametrize("group,dim,S", [(1, 64, 1), (5, 128, 1), (12, 64, 1), (5, 128, 2), (12, 128, 1), (8, 128, 4),
                                         (8, 64, 8), (8, 128, 8), (4, 256, 1), (5, 256, 5)])
def test_visible_infinities(qg, kv, out, group, dim, S):
    check(qg, kv, out, [1, 2, 40, 17, 0, 333], 2, group, dim, S)


@pytest.mark.parametrize("kv,out", [("bf16", "bf16"), ("f16", "f32")])
@pytest.mark.parametrize("group,S", [(5, 1), (8, 4)])
def test_visible_infinities_in_shared_segments(qg, kv, out, group, S):
    """Clusters, and equal ranges joined by a second kernel."""
    check(qg, kv, out, [3000, 20], 2, group, 128, S, page=24)
    check(qg, kv, out, [9000, 500, 3], 1, group, 128, S)
    check(qg, kv, out, [100, 7, 333, 20] * 25, 2, group, 128, S)
