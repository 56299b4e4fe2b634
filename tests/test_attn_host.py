"""Refusals of the attention block's entry points on the host (no GPU): bad
arguments return the named status before any pointer is touched."""
import ctypes
import importlib.util
import os

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
P = 0xDEADBE00          # 256-byte aligned, never mapped: a dereference would fault


@pytest.fixture(scope="module")
def qg():
    spec = importlib.util.spec_from_file_location(
        "qgemv_build", os.path.join(ROOT, "weight_only_quantized_i4g_gb300", "_build.py"))
    build_script = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(build_script)
    build_script.build()
    import weight_only_quantized_i4g_gb300 as m
    return m


def cache(qg, **kw):
    d = dict(k=P, v=P, k_scale=P, v_scale=P, weight=P, page_stride=4 * 16 * 128, head_stride=16 * 128,
             token_stride=128, type=qg.QG_BF16, n_pages=100, page_size=16, n_heads=4, head_dim=128)
    d.update(kw)
    return qg.KVCache(**d)


def append(qg, c=None, **kw):
    d = dict(table=P, table_stride=8, n_seq=2, seq=P, slot=P, T=3, q=P, q_type=qg.QG_BF16, qkv=P, qkv_type=qg.QG_F32,
             qkv_stride=16 * 128, n_q_heads=8, pos=P, n_axes=1, axis=None, inv_freq=P, rotary_dim=128,
             style=qg.QG_ROPE_HALF, stream=0)
    d.update(kw)
    return qg.qg_rope_append(c if c is not None else cache(qg), **d)


def attn(qg, c=None, **kw):
    d = dict(table=P, table_stride=8, lens=P, n_seq=64, max_len=100, o=P, o_type=qg.QG_F32, lse=P, q=P,
             q_type=qg.QG_BF16, q_stride=8 * 128, S=1, n_q_heads=8, scale=0.1, accumulate=0, ws=P, ws_bytes=1 << 40,
             stream=0)
    d.update(kw)
    return qg.qattn_paged(c if c is not None else cache(qg), **d)


def evict(qg, c=None, **kw):
    d = dict(table=P, table_stride=8, dst_table=P, dst_stride=4, lens=P, n_seq=2, max_len=100, budget=64, sinks=4,
             recent=8, kept=P, new_lens=P + 256, stream=0)
    d.update(kw)
    return qg.qg_kv_evict(c if c is not None else cache(qg), **d)


BAD_CACHES = [
    (dict(type=0), "EINVAL"), (dict(type=9), "EINVAL"), (dict(k=None), "EINVAL"), (dict(v=None), "EINVAL"),
    (dict(n_pages=0), "EINVAL"), (dict(page_size=0), "EINVAL"), (dict(n_heads=-1), "EINVAL"),
    (dict(head_dim=0), "ESHAPE"), (dict(head_dim=264), "ESHAPE"), (dict(head_dim=100), "ESHAPE"),
    (dict(type=3, head_dim=72), "ESHAPE"), (dict(type=3, k_scale=None), "EINVAL"), (dict(type=3, v_scale=None), "EINVAL"),
    (dict(k=P + 8), "EALIGN"), (dict(v=P + 2), "EALIGN"), (dict(token_stride=132), "EALIGN"),
    (dict(head_stride=16 * 128 + 4), "EALIGN"), (dict(page_stride=4 * 16 * 128 + 1), "EALIGN"),
    (dict(token_stride=64), "EINVAL"), (dict(page_stride=0), "EINVAL"), (dict(page_stride=1 << 60), "EINVAL"),
    (dict(weight=P + 2), "EALIGN"), (dict(k_scale=P + 1), "EALIGN"),
]


@pytest.mark.parametrize("change,status", BAD_CACHES)
def test_bad_caches(qg, change, status):
    c = cache(qg, **change)
    want = getattr(qg, "QG_" + status)
    assert append(qg, c) == want and attn(qg, c) == want and evict(qg, c) == want
    assert qg.qattn_workspace_bytes(c, 2, 100, 1, 8) == 0


def test_missing_cache(qg):
    n0 = qg.qg_launch_count()
    assert qg.qg_kv_evict(None, P, 8, P, 4, P, 2, 100, 64, 4, 8, P, P, stream=0) == qg.QG_EINVAL
    assert "cache" in qg.last_error()
    assert qg.qg_launch_count() == n0


@pytest.mark.parametrize("change,status", [
    (dict(T=-1), "EINVAL"), (dict(n_q_heads=0), "EINVAL"), (dict(n_q_heads=6), "EINVAL"), (dict(q_type=0), "EINVAL"),
    (dict(q_type=3), "EINVAL"), (dict(qkv_type=3), "EINVAL"), (dict(qkv_stride=16 * 128 - 1), "EINVAL"),
    (dict(rotary_dim=130), "EINVAL"), (dict(rotary_dim=7), "EINVAL"), (dict(rotary_dim=-2), "EINVAL"),
    (dict(style=2), "EINVAL"), (dict(n_axes=0), "EINVAL"), (dict(axis=bytes([0] * 63 + [1])), "EINVAL"),
    (dict(n_seq=0), "EINVAL"), (dict(table=None), "EINVAL"), (dict(table_stride=0), "EINVAL"),
    (dict(seq=None), "EINVAL"), (dict(slot=None), "EINVAL"), (dict(q=None), "EINVAL"), (dict(qkv=None), "EINVAL"),
    (dict(pos=None), "EINVAL"), (dict(inv_freq=None), "EINVAL"), (dict(table=P + 2), "EALIGN"),
    (dict(pos=P + 1), "EALIGN"), (dict(q=P + 1), "EALIGN"), (dict(qkv=P + 2), "EALIGN"),
])
def test_append_refusals(qg, change, status):
    assert append(qg, **change) == getattr(qg, "QG_" + status)


@pytest.mark.parametrize("change,status", [
    (dict(S=0), "EINVAL"), (dict(S=9), "EINVAL"), (dict(n_seq=-1), "EINVAL"), (dict(n_q_heads=5), "EINVAL"),
    (dict(o_type=3), "EINVAL"), (dict(q_type=2), "EINVAL"), (dict(q_type=0), "EINVAL"),
    (dict(q_stride=8 * 128 - 8), "EINVAL"), (dict(scale=float("nan")), "EINVAL"), (dict(scale=float("inf")), "EINVAL"),
    (dict(max_len=-1), "EINVAL"), (dict(max_len=129), "EINVAL"), (dict(table=None), "EINVAL"),
    (dict(lens=None), "EINVAL"), (dict(o=None), "EINVAL"), (dict(q=None), "EINVAL"), (dict(lens=P + 2), "EALIGN"),
    (dict(lse=P + 2), "EALIGN"), (dict(q=P + 8), "EALIGN"), (dict(o=P + 4), "EALIGN"), (dict(q_stride=1028), "EALIGN"),
    (dict(ws=None), "EWORKSPACE"), (dict(ws_bytes=1), "EWORKSPACE"), (dict(ws=P + 16), "EALIGN"),
    (dict(n_seq=1 << 30), "EINVAL"),
])
def test_attention_refusals(qg, change, status):
    assert attn(qg, **change) == getattr(qg, "QG_" + status), qg.last_error()


def test_attention_accumulate_needs_weight(qg):
    assert attn(qg, cache(qg, weight=None), accumulate=1) == qg.QG_EINVAL
    assert "weight" in qg.last_error()
    assert evict(qg, cache(qg, weight=None)) == qg.QG_EINVAL


def test_8_bit_cache_takes_both_query_types(qg):
    """Past the argument checks both are refused for the workspace only."""
    c = cache(qg, type=qg.QG_E4M3)
    for qt in (qg.QG_BF16, qg.QG_F16):
        assert attn(qg, c, q_type=qt, ws=None) == qg.QG_EWORKSPACE


@pytest.mark.parametrize("change,status", [
    (dict(budget=0), "EINVAL"), (dict(sinks=-1), "EINVAL"), (dict(recent=-1), "EINVAL"),
    (dict(sinks=40, recent=25), "EINVAL"), (dict(n_seq=-2), "EINVAL"), (dict(dst_table=None), "EINVAL"),
    (dict(dst_stride=3), "EINVAL"), (dict(max_len=129), "EINVAL"), (dict(lens=None), "EINVAL"),
    (dict(kept=None), "EINVAL"), (dict(new_lens=None), "EINVAL"), (dict(new_lens=P), "EINVAL"),
    (dict(kept=P + 1), "EALIGN"), (dict(dst_table=P + 3), "EALIGN"),
])
def test_evict_refusals(qg, change, status):
    assert evict(qg, **change) == getattr(qg, "QG_" + status), qg.last_error()


def test_nothing_to_do(qg):
    n0 = qg.qg_launch_count()
    assert append(qg, T=0) == qg.QG_OK and attn(qg, n_seq=0) == qg.QG_OK and evict(qg, n_seq=0) == qg.QG_OK
    assert qg.qg_launch_count() == n0


def test_binding_checks_its_tensors(qg):
    torch = pytest.importorskip("torch")
    k = torch.zeros(3, 2, 4, 64, dtype=torch.bfloat16)
    c = qg.kv_cache(k, k.clone(), weight=torch.zeros(3, 2, 4))
    assert (c.n_pages, c.n_heads, c.page_size, c.head_dim) == (3, 2, 4, 64)
    assert (c.page_stride, c.head_stride, c.token_stride, c.type) == (512, 256, 64, qg.QG_BF16)
    c = qg.kv_cache(k, k.clone(), order="token")
    assert (c.n_heads, c.page_size, c.head_stride, c.token_stride) == (4, 2, 64, 256)
    for bad in (dict(v=k.half()), dict(v=k[:2]), dict(order="x"), dict(weight=torch.zeros(3, 4, 2)),
                dict(k=k.float(), v=k.float()), dict(k_scale=torch.zeros(3)), dict(k=k[..., ::2], v=k[..., ::2])):
        a = dict(k=k, v=k)
        a.update(bad)
        with pytest.raises(ValueError):
            qg.kv_cache(**a)
    with pytest.raises(ValueError):
        append(qg, axis=bytes(63))
    assert ctypes.sizeof(qg.KVCache) == 8 * 8 + 5 * 4 + 4
    assert qg.strerror(qg.QG_EPAGE).startswith("QG_EPAGE")
