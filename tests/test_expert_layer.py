"""The expert layer's operators together, as the example runs them: every stage
against its definition in 64 bits on what the stage before it left, the layer
captured into a graph and replayed on other tokens, and the gradients of a
trained layer's tokens, experts and router."""
import os
import sys

import pytest

torch = pytest.importorskip("torch")

from moe_util import HALF, TINY, U, codes_of, product, routing, sorted_slots  # noqa: E402

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def ex():
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    import expert_layer as m
    return m


def randn(seed, *shape):
    return torch.randn(*shape, generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda")


def make(ex, tokens=70, experts=6, hidden=400, width=272, top=3):
    return ex.ExpertLayer(randn(1, experts, 2 * width, hidden) * hidden ** -0.5, randn(2, experts, hidden, width) * width ** -0.5,
                          tokens, top)


def slots(tokens, top, experts, seed, away):
    ids = routing(tokens, top, experts, seed, away)
    return ids, torch.tensor(ids, dtype=torch.int32, device="cuda"), torch.softmax(randn(seed, tokens, top), 1)


@pytest.mark.parametrize("tokens,hidden,width,away", [(70, 400, 272, 0.0), (1, 400, 272, 0.0), (64, 256, 130 * 8, 0.3),
                                                      (700, 1024, 384, 0.1), (33, 304, 144, 1.0)])
def test_every_stage(ex, tokens, hidden, width, away):
    layer = make(ex, tokens, hidden=hidden, width=width)
    x = randn(3, tokens, hidden).bfloat16()
    lists, ids, weights = slots(tokens, 3, 6, 4, away)
    out = torch.full_like(x, 7.0)
    layer(out, x, ids, weights)
    torch.cuda.synchronize()
    offsets, order, place = sorted_slots(lists, 6)
    n = len(order)
    assert layer.offsets.tolist() == offsets and layer.place.tolist() == place
    codes, scale = codes_of(x)
    slot = torch.tensor(order, dtype=torch.long)
    assert torch.equal(layer.x[:n].view(torch.uint8).cpu(), codes.view(torch.uint8)[slot // 3])
    assert torch.equal(layer.x_scale[:n].cpu(), scale[slot // 3])
    # products: 1e-3 of the magnitudes, and bf16's rounding
    for got, a, sa, w, sw in ((layer.gu, layer.x, layer.x_scale, layer.up, layer.up_scale),
                              (layer.y, layer.a, layer.a_scale, layer.down, layer.down_scale)):
        want, mag = product(a[:n], sa[:n], w, sw, offsets)
        assert bool(((got[:n].double() - want).abs() <= 1e-3 * mag * (1 + HALF["bf16"]) + HALF["bf16"] * want.abs() + TINY["bf16"]).all())
    codes, scale = codes_of(layer.act[:n])
    assert torch.equal(layer.a[:n].view(torch.uint8).cpu(), codes.view(torch.uint8))
    assert torch.equal(layer.a_scale[:n].cpu(), scale)
    p = torch.tensor(place, device="cuda").view(tokens, 3)
    r = layer.y.double()[p.clamp_min(0)] * torch.where(p >= 0, weights.double(), 0.0)[..., None]
    r = torch.where((p >= 0)[..., None], r, 0.0)
    slack = 4 * U * r.abs().sum(1)
    err = (out.double() - r.sum(1)).abs()
    assert bool((err <= slack + HALF["bf16"] * (r.sum(1).abs() + slack) + TINY["bf16"]).all())
    import weight_only_quantized_i4g_gb300 as qg
    assert qg.qg_device_status() == (0, 0)


def test_captured_and_replayed_on_other_tokens(ex):
    layer, twin = make(ex, 200), make(ex, 200)
    x, out = torch.zeros(200, 400, dtype=torch.bfloat16, device="cuda"), torch.zeros(200, 400, dtype=torch.bfloat16, device="cuda")
    ids, weights = torch.zeros(200, 3, dtype=torch.int32, device="cuda"), torch.zeros(200, 3, device="cuda")
    layer(out, x, ids, weights)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        layer(out, x, ids, weights)
    for seed in range(5):
        x.copy_(randn(10 + seed, 200, 400))
        _, i, w = slots(200, 3, 6, 20 + seed, 0.1 * seed)
        if seed == 3:
            i.fill_(4)                                      # everything to one expert
        ids.copy_(i)
        weights.copy_(w)
        graph.replay()
        want = torch.empty_like(out)
        twin(want, x, ids, weights)
        torch.cuda.synchronize()
        assert torch.equal(out, want), seed


def test_fewer_tokens_than_the_layer_holds(ex):
    layer = make(ex, 3000)
    for tokens in (3000, 1, 1400, 17):
        x = randn(3, tokens, 400).bfloat16()
        _, ids, weights = slots(tokens, 3, 6, 4, 0.1)
        out, want = torch.empty_like(x), torch.empty_like(x)
        layer(out, x, ids, weights)
        make(ex, tokens)(want, x, ids, weights)
        torch.cuda.synchronize()
        # Another number of rows may choose another kernel, whose sums go in another order, 2^-20 or so apart.  About
        # one value in 4000 then rounds to the other bf16 neighbour (2^-8), one in 16 of those to another code (2^-4):
        # with one such code among a token's 3 x 272, its row moves by 2^-4 / sqrt(272) = 0.4%, with four by 0.8%
        err = (out.double() - want.double()).norm(dim=1)
        assert bool((err <= 1e-2 * want.double().norm(dim=1)).all())


def test_gradients_of_a_trained_layer(ex):
    """f32 throughout: dispatch, an expert's product each, combine; against autograd in 64 bits."""
    tokens, top, experts, hidden = 41, 3, 5, 52
    lists, _, _ = slots(tokens, top, experts, 9, 0.15)
    offsets, order, place = sorted_slots(lists, experts)
    n = len(order)
    pl = torch.tensor(place, dtype=torch.int32, device="cuda").view(tokens, top)
    base = [randn(1, tokens, hidden), randn(2, experts, hidden, hidden) * hidden ** -0.5, torch.softmax(randn(3, tokens, top), 1)]
    dout = randn(4, tokens, hidden)

    def run(x, w, weights, wide):
        if wide:
            slot = torch.tensor(order, device="cuda")
            rows = x[slot // top]
        else:
            rows = ex.Dispatch.apply(x, pl, n)
        y = torch.cat([rows[offsets[e]:offsets[e + 1]] @ w[e].t() for e in range(experts)])
        if wide:
            out = torch.zeros(tokens, hidden, dtype=torch.float64, device="cuda")
            return out.index_add(0, slot // top, y * weights.reshape(-1)[slot][:, None])
        return ex.Combine.apply(y, weights, pl)
    sides = []
    for wide in (False, True):
        leaves = [(b.double() if wide else b.clone()).requires_grad_() for b in base]
        out = run(*leaves, wide)
        out.backward(dout.double() if wide else dout)
        sides.append([out.detach()] + [leaf.grad for leaf in leaves])
    mags = [b.abs().double().requires_grad_() for b in base]                # the same sums of magnitudes
    out = run(*mags, True)
    out.backward(dout.abs().double())
    # a value is a sum of products of at most four f32 factors: two sums over `hidden` and two over `top` or a group's
    # rows on its way (each at most n long), every addition and product off by half a step
    terms = 2 * hidden + 2 * max(top, n) + 8
    for got, want, mag in zip(*sides, [out.detach()] + [m.grad for m in mags]):
        assert bool(((got.double() - want).abs() <= terms * U * mag + 1e-40).all())
