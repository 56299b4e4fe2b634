"""Attention weights of drafted tokens' slots where some row is NaN: a slot
takes weight only from the rows that see it."""
import pytest

torch = pytest.importorskip("torch")

from attn_util import DEV, Paged, attention, run_attention  # noqa: E402
from test_attn_paged import queries  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def qg():
    import weight_only_quantized_i4g_gb300 as m
    return m


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("kv", ["bf16", "f16", "e4m3"])
@pytest.mark.parametrize("S,group,dim,lens", [(2, 1, 64, [20, 33, 1]), (4, 5, 128, [130, 2, 700, 4]),
                                              (8, 9, 128, [40, 7, 300]), (4, 6, 256, [50, 3])])
def test_rows_of_nan_leave_hidden_slots_alone(qg, bad, kv, S, group, dim, lens):
    """Token 0's queries hold NaN or infinity: of its sequence's slots only those
    that it does not see keep finite weights."""
    pc = Paged(qg, lens, 2, dim, kv, seed=S + group, weight=True).fill()
    q = queries(pc, len(lens), S, 2 * group, kv)
    q.view(len(lens), S, -1)[:, 0] = bad
    before = pc.weight.double()
    run_attention(pc, q, S, 2 * group, dim ** -0.5, accumulate=True)
    torch.cuda.synchronize()
    assert qg.qg_device_status() == (0, 0)
    clean = q.clone()
    clean.view(len(lens), S, -1)[:, 0] = 0.0         # token 0 draws on no slot that is checked below
    w64 = attention(pc, clean, S, 2 * group, dim ** -0.5)[2]
    for b, n in enumerate(lens):
        seen = max(n - S + 1, 0)                     # slots that token 0 sees
        for h in range(2):
            p, i = pc.where(b)
            got = pc.weight[p, h, i].double()
            assert bool(torch.isnan(got[:seen]).all())
            want = before[p, h, i] + w64[b, h]
            assert float((got[seen:] - want[seen:]).abs().max()) < 1e-3, (b, h)
