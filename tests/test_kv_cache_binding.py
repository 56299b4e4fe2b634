"""Strides that the cache's binding takes from its tensors (host only)."""
import pytest

from test_attn_host import attn, evict, qg  # noqa: F401

torch = pytest.importorskip("torch")


def strided(shape, strides):
    size = sum((n - 1) * s for n, s in zip(shape, strides)) + 1
    return torch.zeros(size, dtype=torch.bfloat16).as_strided(shape, strides)


@pytest.mark.parametrize("shape,k,v", [
    ((5, 1, 16, 64), (1024, 1, 64, 1), (1024, 1024, 64, 1)),       # one head
    ((5, 2, 1, 64), (128, 64, 1, 1), (128, 64, 0, 1)),             # one slot a page
    ((1, 2, 16, 64), (7, 1024, 64, 1), (2048, 1024, 64, 1)),       # one page
    ((1, 1, 1, 64), (0, 0, 0, 1), (64, 64, 64, 1)),
])
@pytest.mark.parametrize("order", ["head", "token"])
def test_axes_of_one_element_have_no_stride(qg, shape, k, v, order):  # noqa: F811
    """k and v lie alike, whatever their strides along such an axis say, and the
    library takes them (these calls end at the first check after the cache's)."""
    c = qg.kv_cache(strided(shape, k), strided(shape, v), weight=torch.zeros(shape[0], shape[1], shape[2])
                    if order == "head" else torch.zeros(shape[0], shape[2], shape[1]), order=order)
    for n, got, a, b in zip(shape, (c.page_stride, c.head_stride if order == "head" else c.token_stride,
                                    c.token_stride if order == "head" else c.head_stride), k, v):
        assert got >= 64 and (n == 1 or got == a == b)
    assert attn(qg, c, S=0) == qg.QG_EINVAL and "S = 0" in qg.last_error()
    assert evict(qg, c, budget=0) == qg.QG_EINVAL and "budget" in qg.last_error()


def test_real_differences_are_refused(qg):  # noqa: F811
    with pytest.raises(ValueError):
        qg.kv_cache(strided((5, 1, 16, 64), (1024, 1024, 64, 1)), strided((5, 1, 16, 64), (2048, 1024, 64, 1)))
    with pytest.raises(ValueError):
        qg.kv_cache(torch.zeros(5, 16, 64, dtype=torch.bfloat16), torch.zeros(5, 16, 64, dtype=torch.bfloat16))
