"""Refusals of the expert layer's entry points, on the host alone: no pointer
is touched and nothing is launched."""
import pytest

from test_abi_host import POISON as P, qg  # noqa: F401


def test_sort_refusals(qg):  # noqa: F811
    def call(offsets=P, order=P, place=P, ids=P, n=4, k=2, e=8, ws=P, wb=1 << 30):
        return qg.qg_moe_sort(offsets, order, place, ids, n, k, e, ws, wb, stream=0)
    before = qg.qg_launch_count()
    assert call(offsets=0) == qg.QG_EINVAL
    assert call(place=0) == qg.QG_EINVAL
    assert call(ids=0) == qg.QG_EINVAL
    assert call(n=-1) == qg.QG_EINVAL
    assert call(k=0) == qg.QG_EINVAL
    assert call(e=0) == qg.QG_EINVAL
    assert call(e=8193) == qg.QG_EINVAL and "8193" in qg.last_error()
    assert call(n=1 << 30, k=2) == qg.QG_EINVAL
    assert call(offsets=P + 2) == qg.QG_EALIGN
    assert call(order=P + 1) == qg.QG_EALIGN
    assert call(ids=P + 2) == qg.QG_EALIGN
    assert call(ws=P + 16) == qg.QG_EALIGN
    need = qg.qg_moe_sort_workspace_bytes(1 << 20, 8, 256)
    if need:
        assert call(n=1 << 20, k=8, e=256, ws=0, wb=0) == qg.QG_EWORKSPACE
        assert call(n=1 << 20, k=8, e=256, wb=need - 1) == qg.QG_EWORKSPACE and str(need) in qg.last_error()
    assert qg.qg_moe_sort_workspace_bytes(-1, 2, 8) == 0
    assert qg.qg_moe_sort_workspace_bytes(4, 2, 8193) == 0
    assert qg.qg_launch_count() == before


def test_dispatch_refusals(qg):  # noqa: F811
    def call(rows=P, rt=qg.QG_BF16, sc=P, x=P, xt=qg.QG_BF16, stride=256, place=P, n=4, k=2, w=256, nr=8):
        return qg.qg_moe_dispatch(rows, rt, sc, x, xt, stride, place, n, k, w, nr, stream=0)
    before = qg.qg_launch_count()
    assert call(rows=0) == qg.QG_EINVAL
    assert call(x=0) == qg.QG_EINVAL
    assert call(rt=qg.QG_E4M3, sc=0) == qg.QG_EINVAL
    assert call(rt=qg.QG_F32) == qg.QG_EINVAL           # a copy keeps its type
    assert call(xt=qg.QG_E4M3, rt=qg.QG_E4M3) == qg.QG_EINVAL
    assert call(xt=9) == qg.QG_EINVAL
    assert call(stride=255) == qg.QG_EINVAL
    assert call(stride=1 << 41) == qg.QG_EINVAL
    assert call(n=-1) == qg.QG_EINVAL
    assert call(nr=-1) == qg.QG_EINVAL
    assert call(k=0) == qg.QG_EINVAL
    assert call(w=0) == qg.QG_EINVAL
    assert call(n=1 << 30, k=2) == qg.QG_EINVAL
    assert call(n=(1 << 31) - 1, k=1, w=129) == qg.QG_EINVAL
    assert call(place=0, nr=7) == qg.QG_EINVAL and "7" in qg.last_error()
    assert call(rows=P + 1) == qg.QG_EALIGN
    assert call(x=P + 1) == qg.QG_EALIGN
    assert call(place=P + 2) == qg.QG_EALIGN
    assert call(rt=qg.QG_E4M3, sc=P + 2) == qg.QG_EALIGN
    assert call(n=0) == qg.QG_OK                        # nothing to do
    assert call(nr=0) == qg.QG_OK
    assert qg.qg_launch_count() == before


def test_combine_refusals(qg):  # noqa: F811
    def call(out=P, ot=qg.QG_BF16, y=P, yt=qg.QG_F32, wt=P, place=P, n=4, k=2, w=256, nr=8):
        return qg.qg_moe_combine(out, ot, y, yt, wt, place, n, k, w, nr, stream=0)
    before = qg.qg_launch_count()
    assert call(out=0) == qg.QG_EINVAL
    assert call(y=0) == qg.QG_EINVAL
    assert call(ot=qg.QG_E4M3) == qg.QG_EINVAL
    assert call(yt=qg.QG_E4M3) == qg.QG_EINVAL
    assert call(place=0, nr=7) == qg.QG_EINVAL
    assert call(k=-3) == qg.QG_EINVAL
    assert call(w=0) == qg.QG_EINVAL
    assert call(out=P + 1) == qg.QG_EALIGN
    assert call(y=P + 2) == qg.QG_EALIGN
    assert call(wt=P + 2) == qg.QG_EALIGN
    assert call(n=0) == qg.QG_OK
    assert qg.qg_launch_count() == before


def test_combine_grad_refusals(qg):  # noqa: F811
    def call(dy=P, dw=P, do=P, dt=qg.QG_BF16, y=P, yt=qg.QG_F32, wt=P, place=P, n=4, k=2, w=256, nr=8):
        return qg.qg_moe_combine_grad(dy, dw, do, dt, y, yt, wt, place, n, k, w, nr, stream=0)
    before = qg.qg_launch_count()
    assert call(dy=0, dw=0) == qg.QG_EINVAL
    assert call(do=0) == qg.QG_EINVAL
    assert call(y=0) == qg.QG_EINVAL
    assert call(dt=qg.QG_E4M3) == qg.QG_EINVAL
    assert call(yt=-1) == qg.QG_EINVAL
    assert call(place=0, nr=7) == qg.QG_EINVAL
    assert call(dy=P + 2) == qg.QG_EALIGN
    assert call(dw=P + 2) == qg.QG_EALIGN
    assert call(do=P + 1) == qg.QG_EALIGN
    assert call(n=0) == qg.QG_OK
    assert qg.qg_launch_count() == before


@pytest.mark.parametrize("grouped", [False, True])
def test_product_refusals(qg, grouped):  # noqa: F811
    def call(fmt=qg.QG_FMT_FP8B128, y=P, yt=qg.QG_BF16, x=P, xs=P, w=P, ws=P, off=P, e=4, m=64, i=256, o=256, wk=P,
             wb=1 << 40):
        if grouped:
            return qg.qgemm_e4m3_moe(fmt, y, yt, x, xs, w, ws, off, e, m, i, o, wk, wb, stream=0)
        return qg.qgemm_e4m3(fmt, y, yt, x, xs, w, ws, m, i, o, wk, wb, stream=0)
    before = qg.qg_launch_count()
    assert call(fmt=qg.QG_FMT_I4G) == qg.QG_EINVAL
    assert call(yt=qg.QG_E4M3) == qg.QG_EINVAL
    for name in ("y", "x", "xs", "w", "ws"):
        assert call(**{name: 0}) == qg.QG_EINVAL, name
    assert call(m=-1) == qg.QG_EINVAL
    assert call(m=65535 * 64 + 1) == qg.QG_EINVAL
    assert call(i=0) == qg.QG_EINVAL
    assert call(o=0) == qg.QG_EINVAL
    assert call(y=P + 1) == qg.QG_EALIGN
    assert call(yt=qg.QG_F32, y=P + 2) == qg.QG_EALIGN
    assert call(xs=P + 2) == qg.QG_EALIGN
    assert call(ws=P + 2) == qg.QG_EALIGN
    assert call(wk=P + 16) == qg.QG_EALIGN
    if grouped:
        assert call(off=0) == qg.QG_EINVAL
        assert call(off=P + 2) == qg.QG_EALIGN
        assert call(e=0) == qg.QG_EINVAL
        assert call(e=8193) == qg.QG_EINVAL
    need = qg.qgemm_e4m3_workspace_bytes(64, 256, 256, 4 if grouped else 1)
    if need:
        assert call(wk=0, wb=0) == qg.QG_EWORKSPACE
        assert call(wb=need - 1) == qg.QG_EWORKSPACE and str(need) in qg.last_error()
    assert call(m=0) == qg.QG_OK
    assert qg.qgemm_e4m3_workspace_bytes(64, 0, 256) == 0
    assert qg.qg_launch_count() == before


@pytest.mark.parametrize("e", [1, 7, 64, 256, 1000, 8192])
def test_sort_workspace_of_more_slots_serves_fewer(qg, e):  # noqa: F811
    sizes = [qg.qg_moe_sort_workspace_bytes(n, 1, e) for n in [1, 1024, 1025, 5000, 100000] + list(range(900000, 1200000, 777)) +
             [2 ** 31 - 1]]
    assert sizes == sorted(sizes)
