"""The example's decode loop (packed projections, cache write, attention,
eviction) against the same steps in 64 bits, through several evictions."""
import os
import sys

import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_decode_loop_matches_plain_steps():
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    import decode_attention as ex
    import weight_only_quantized_i4g_gb300 as qg

    g = torch.Generator(device="cuda").manual_seed(3)
    hidden, hq, hkv, dim, batch, budget = 512, 6, 2, 64, 3, 40
    w_qkv = torch.randn((hq + 2 * hkv) * dim, hidden, generator=g, device="cuda") * hidden ** -0.5
    w_o = torch.randn(hidden, hq * dim, generator=g, device="cuda") * (hq * dim) ** -0.5
    block = ex.AttentionBlock(w_qkv, w_o, batch, hq, hkv, dim, budget, page=8, sinks=2, recent=8)

    def dense(p):            # the packed weights' values
        nib = torch.stack([p.q & 15, p.q >> 4], -1).reshape(p.O, p.I).double() - 8
        return nib * p.scales.double().repeat_interleave(ex.GROUP, 1)

    wq, wo = dense(block.qkv), dense(block.out)
    keys = [[torch.zeros(0, dim, dtype=torch.float64, device="cuda") for _ in range(hkv)] for _ in range(batch)]
    vals = [[k.clone() for k in row] for row in keys]
    evictions = 0
    for step in range(120):
        x = torch.randn(batch, hidden, generator=g, device="cuda")
        before = block.length
        y = block.step(x).clone()
        if block.length <= before:                   # this step began with an eviction
            evictions += 1
            for b in range(batch):
                for h in range(hkv):
                    at = block.kept[b, h].long()
                    keys[b][h], vals[b][h] = keys[b][h][at], vals[b][h][at]
        qkv = (x.double() @ wq.T).view(batch, hq + 2 * hkv, dim)
        a = step * block.inv_freq.double()
        lo, hi = qkv[..., :dim // 2], qkv[..., dim // 2:]
        turned = torch.cat([lo * a.cos() - hi * a.sin(), hi * a.cos() + lo * a.sin()], -1)
        o = torch.zeros(batch, hq, dim, dtype=torch.float64, device="cuda")
        for b in range(batch):
            for h in range(hkv):
                keys[b][h] = torch.cat([keys[b][h], turned[b, hq + h].bfloat16().double()[None]])
                vals[b][h] = torch.cat([vals[b][h], qkv[b, hq + hkv + h].bfloat16().double()[None]])
                rows = slice(h * hq // hkv, (h + 1) * hq // hkv)
                z = turned[b, rows].bfloat16().double() @ keys[b][h].T * dim ** -0.5
                o[b, rows] = torch.softmax(z, -1) @ vals[b][h]
        want = o.view(batch, -1) @ wo.T
        # q, k, v are bf16 on both sides, from projections 1e-3 apart at most: a
        # value on a rounding edge may differ by 2^-8, so 1% of the output's size
        assert float((y.double() - want).norm() / want.norm()) < 1e-2, step
    assert evictions >= 8 and block.length <= budget + 8
    assert qg.qg_device_status() == (0, 0)
    assert sorted(block.free + [p for t in block.tables for p in t]) == list(range(block.k.shape[0]))
