"""What the expert-layer example refuses, on the host: the library gets
addresses alone, so types, shapes and layouts are looked at before a call."""
import os
import sys

import pytest

torch = pytest.importorskip("torch")

from test_abi_host import qg  # noqa: F401

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture()
def ex(qg, monkeypatch):  # noqa: F811
    """The example, with every entry point that would launch replaced by one that counts."""
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    import expert_layer as m
    m.calls = []
    for name in ("qg_moe_sort", "qg_moe_dispatch", "qg_moe_combine", "qg_moe_combine_grad", "qgemm_e4m3_moe"):
        monkeypatch.setattr(qg, name, lambda *a, _n=name: m.calls.append(_n) or 0)
    return m


def layer_args(t=4, h=32, k=2):
    return [torch.zeros(t, h, dtype=torch.bfloat16), torch.zeros(t, h, dtype=torch.bfloat16),
            torch.zeros(t, k, dtype=torch.int32), torch.zeros(t, k)]


def test_layer_refuses_what_it_cannot_take(ex):
    layer = ex.ExpertLayer(torch.ones(3, 32, 32), torch.ones(3, 32, 16), 4, 2)
    good = layer_args()
    layer(*good)
    assert len(ex.calls) == 6
    layer(*layer_args(t=1))
    layer(good[0], torch.zeros(4, 40, dtype=torch.bfloat16)[:, :32], *good[2:])      # rows further apart
    assert len(ex.calls) == 18
    bad = [layer_args(t=5)]                                              # more tokens than places
    for at, wrong in ((0, good[0].float()), (0, good[0][:3]), (0, good[0].t().contiguous().t()),
                      (1, good[1].half()), (1, torch.zeros(4, 64, dtype=torch.bfloat16)[:, ::2]), (1, good[1][:, :16]),
                      (2, good[2].long()), (2, torch.zeros(2, 4, dtype=torch.int32).t()), (2, good[2][:, :1]),
                      (3, good[3].bfloat16()), (3, good[3][:2]), (3, torch.zeros(2, 4).t())):
        bad.append(good[:at] + [wrong] + good[at + 1:])
    for args in bad:
        with pytest.raises(ValueError):
            layer(*args)
    assert len(ex.calls) == 18


@pytest.mark.parametrize("place,weights", [
    (torch.zeros(4, 2, dtype=torch.int64), torch.zeros(4, 2)),           # torch's own index type
    (torch.zeros(2, 4, dtype=torch.int32).t(), torch.zeros(4, 2)),
    (torch.zeros(8, dtype=torch.int32), torch.zeros(8)),
    (torch.zeros(4, 2, dtype=torch.int32), torch.zeros(4, 2, dtype=torch.bfloat16)),
    (torch.zeros(4, 2, dtype=torch.int32), torch.zeros(4, 3)),
    (torch.zeros(4, 2, dtype=torch.int32), torch.zeros(3, 2))])
def test_wrappers_refuse_other_places_and_weights(ex, place, weights):
    with pytest.raises(ValueError):
        ex.Combine.apply(torch.zeros(8, 16), weights, place)
    if place.dtype != torch.int32 or place.dim() != 2 or not place.is_contiguous():
        with pytest.raises(ValueError):
            ex.Dispatch.apply(torch.zeros(4, 16), place, 8)
    with pytest.raises(ValueError):
        ex.Dispatch.apply(torch.zeros(3, 16), place, 8)                  # places of other tokens
    assert ex.calls == []


def test_wrappers_take_places_and_weights(ex):
    place = torch.zeros(4, 2, dtype=torch.int32)
    assert ex.Combine.apply(torch.zeros(8, 16), torch.zeros(2, 4).t(), place).shape == (4, 16)
    assert ex.Dispatch.apply(torch.zeros(16, 4).t(), place, 8).shape == (8, 16)
    assert len(ex.calls) == 2


@pytest.mark.parametrize("wrapper", ["dispatch", "combine"])
def test_second_derivatives_are_refused(ex, wrapper):
    """Where another path carries the graph, a second derivative through the wrapper would be left out without a word."""
    place = torch.zeros(4, 2, dtype=torch.int32)
    if wrapper == "dispatch":
        x = torch.ones(4, 16, requires_grad=True)
        y = ex.Dispatch.apply(x, place, 8)
    else:
        x = torch.ones(8, 16, requires_grad=True)
        y = ex.Combine.apply(x, torch.zeros(4, 2), place)
    first, = torch.autograd.grad(y.square().sum() + x.pow(3).sum(), x, create_graph=True)
    with pytest.raises(RuntimeError, match="once_differentiable"):
        first.sum().backward()


@pytest.mark.parametrize("rows,router", [(True, True), (True, False), (False, True)])
def test_only_the_gradients_wanted_are_asked_for(ex, qg, monkeypatch, rows, router):  # noqa: F811
    asked = []
    monkeypatch.setattr(qg, "qg_moe_combine_grad", lambda dy, dw, *a: asked.append((dy is not None, dw is not None)) or 0)
    y, weights = torch.ones(8, 16, requires_grad=rows), torch.ones(4, 2, requires_grad=router)
    ex.Combine.apply(y, weights, torch.zeros(4, 2, dtype=torch.int32)).sum().backward()
    assert asked == [(rows, router)]
    assert (y.grad is not None, weights.grad is not None) == (rows, router)
