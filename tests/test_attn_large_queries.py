"""Attention over an 8-bit cache with queries from the smallest bf16 numbers to
the largest: each row is scaled into f16's range by a power of two."""
import pytest

torch = pytest.importorskip("torch")

from attn_util import Paged, check_attention  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def qg():
    import weight_only_quantized_i4g_gb300 as m
    return m


@pytest.mark.parametrize("exponent", [-133, -126, -120, -100, -50, 0, 50, 100, 114, 115, 118, 122, 126])
def test_queries_of_any_size(qg, exponent):
    """Rows of 2^exponent and a scale of 8 * 2^-exponent, as far as f32 has it."""
    pc = Paged(qg, [70, 5, 260], 2, 64, "e4m3", seed=6).fill(1.0)
    # codes of 1 and scales of 2^-6: no sum passes f32's range at 2^127
    q = pc.randn(3, 8 * 64).clamp(-1.9, 1.9)
    if exponent < -126:
        q = q.sign()                                  # subnormal: whole bits only
    q = (q.double() * 2.0 ** exponent).bfloat16()
    assert bool(torch.isfinite(q).all()) and bool((q != 0).any())
    pc.k_scale.fill_(2.0 ** -6)
    check_attention(pc, q, 1, 8, 8.0 * 2.0 ** min(-exponent, 120))
