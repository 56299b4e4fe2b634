"""The attention block of a decode loop on packed weights and a bounded cache.

For every step and every sequence of a small batch:

    qkv = W_qkv x            qgemv_i4g (grouped int4, f32 activations)
    q, cache <- rope(qkv)    qg_rope_append
    o = attention(q, cache)  qattn_paged, adding up each slot's weight
    y = W_o o                qgemv_i4g

and, whenever the caches pass their budget by a page, qg_kv_evict copies the
slots worth keeping to fresh pages and the old pages return to the pool.

    python examples/decode_attention.py [--steps 2000] [--budget 512]
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import weight_only_quantized_i4g_gb300 as qg  # noqa: E402

GROUP = 64      # int4 group size


class PackedLinear:
    """f32 weights [O, I] packed to grouped int4 on the device."""

    def __init__(self, w: torch.Tensor):
        self.O, self.I = w.shape
        self.q = torch.empty(self.O, self.I // 2, dtype=torch.uint8, device=w.device)
        self.scales = torch.empty(self.O, self.I // GROUP, device=w.device)
        qg.check(qg.qg_quantize_i4g(self.q, self.scales, w, self.O, self.I, GROUP))
        self.ws_bytes = qg.qg_workspace_bytes(qg.QG_FMT_I4G, 8, self.I, self.O, GROUP)
        self.ws = torch.empty(max(self.ws_bytes, 1), dtype=torch.uint8, device=w.device)

    def __call__(self, y: torch.Tensor, x: torch.Tensor) -> None:
        qg.check(qg.qgemv_i4g(y, x, self.q, self.scales, x.shape[0], self.I, self.O, GROUP, self.ws, self.ws_bytes))


class AttentionBlock:
    """One attention block over `batch` sequences whose caches hold at most
    `budget` slots a head, or a page more between two evictions."""

    def __init__(self, w_qkv, w_o, batch, q_heads, kv_heads, dim, budget, page=16, sinks=4, recent=64, theta=1e4):
        dev = w_qkv.device
        self.batch, self.q_heads, self.kv_heads, self.dim = batch, q_heads, kv_heads, dim
        self.budget, self.page, self.recent = budget, page, min(recent, budget // 2)
        self.sinks = min(sinks, budget - self.recent)
        self.qkv, self.out = PackedLinear(w_qkv), PackedLinear(w_o)
        self.limit = budget + page                               # slots at which the caches are cut
        self.width = -(-self.limit // page)                      # pages of a sequence
        kept_pages = -(-budget // page)
        pages = batch * (self.width + kept_pages)                # room for the survivors beside the old pages
        shape = (pages, kv_heads, page, dim)
        self.k = torch.zeros(shape, dtype=torch.bfloat16, device=dev)
        self.v = torch.zeros_like(self.k)
        self.weight = torch.zeros(pages, kv_heads, page, device=dev)
        self.cache = qg.kv_cache(self.k, self.v, weight=self.weight)
        self.free = list(range(pages))
        self.tables = [[] for _ in range(batch)]                 # pages of each sequence (host)
        self.table = torch.full((batch, self.width), -1, dtype=torch.int32, device=dev)
        self.lens = torch.zeros(batch, dtype=torch.int32, device=dev)
        self.length = 0                                          # slots in use, the same for all sequences here
        self.tokens = 0                                          # tokens seen: their positions
        self.seq = torch.arange(batch, dtype=torch.int32, device=dev)
        self.inv_freq = (theta ** (-torch.arange(0, dim, 2, dtype=torch.float64) / dim)).float().to(dev)
        self.y_qkv = torch.empty(batch, (q_heads + 2 * kv_heads) * dim, device=dev)
        self.q = torch.empty(batch, q_heads * dim, dtype=torch.bfloat16, device=dev)
        self.o = torch.empty(batch, q_heads * dim, device=dev)
        self.y = torch.empty(batch, self.out.O, device=dev)
        self.ws_bytes = qg.qattn_workspace_bytes(self.cache, batch, self.width * page, 1, q_heads, 1)
        self.ws = torch.empty(max(self.ws_bytes, 1), dtype=torch.uint8, device=dev)
        self.kept = torch.empty(batch, kv_heads, budget, dtype=torch.int32, device=dev)
        self.new_lens = torch.empty_like(self.lens)

    def _upload(self):
        rows = [t + [-1] * (self.width - len(t)) for t in self.tables]
        self.table.copy_(torch.tensor(rows, dtype=torch.int32))

    def evict(self):
        """Cut every cache to the budget on fresh pages."""
        fresh = [[self.free.pop() for _ in range(-(-self.budget // self.page))] for _ in range(self.batch)]
        dst = torch.tensor(fresh, dtype=torch.int32, device=self.table.device)
        qg.check(qg.qg_kv_evict(self.cache, self.table, self.width, dst, dst.shape[1], self.lens, self.batch,
                                self.width * self.page, self.budget, self.sinks, self.recent, self.kept, self.new_lens))
        for old in self.tables:
            self.free.extend(old)
        self.tables = fresh
        self.lens.copy_(self.new_lens)
        self.length = min(self.length, self.budget)
        self._upload()

    def step(self, x: torch.Tensor) -> torch.Tensor:
        """One token per sequence: x f32 [batch, I] -> y f32 [batch, O]."""
        if self.length == self.limit:
            self.evict()
        if self.length == len(self.tables[0]) * self.page:
            for t in self.tables:
                t.append(self.free.pop())
            self._upload()
        slot = self.lens.clone()
        pos = torch.full((self.batch, 1), self.tokens, dtype=torch.int32, device=x.device)
        self.lens += 1
        self.length += 1
        self.tokens += 1
        self.qkv(self.y_qkv, x)
        qg.check(qg.qg_rope_append(self.cache, self.table, self.width, self.batch, self.seq, slot, self.batch, self.q,
                                   qg.QG_BF16, self.y_qkv, qg.QG_F32, self.y_qkv.shape[1], self.q_heads, pos, 1, None,
                                   self.inv_freq, self.dim, qg.QG_ROPE_HALF))
        qg.check(qg.qattn_paged(self.cache, self.table, self.width, self.lens, self.batch, self.width * self.page,
                                self.o, qg.QG_F32, None, self.q, qg.QG_BF16, self.q.shape[1], 1, self.q_heads,
                                self.dim ** -0.5, 1, self.ws, self.ws_bytes))
        self.out(self.y, self.o)
        return self.y


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--steps", type=int, default=2000)
    ap.add_argument("--batch", type=int, default=4)
    ap.add_argument("--hidden", type=int, default=5120)
    ap.add_argument("--budget", type=int, default=512)
    a = ap.parse_args()
    g = torch.Generator(device="cuda").manual_seed(0)
    dim, q_heads, kv_heads = 128, a.hidden // 128, 8
    w_qkv = torch.randn((q_heads + 2 * kv_heads) * dim, a.hidden, generator=g, device="cuda") * a.hidden ** -0.5
    w_o = torch.randn(a.hidden, q_heads * dim, generator=g, device="cuda") * a.hidden ** -0.5
    block = AttentionBlock(w_qkv, w_o, a.batch, q_heads, kv_heads, dim, a.budget)
    x = torch.randn(a.batch, a.hidden, generator=g, device="cuda")
    begin, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    for i in range(a.steps):
        if i == a.steps // 10:
            begin.record()
        y = block.step(x)
        x = torch.nn.functional.normalize(x + y, dim=-1) * a.hidden ** 0.5
    end.record()
    torch.cuda.synchronize()
    rc, status = qg.qg_device_status()
    qg.check(rc)
    qg.check(status)
    n = a.steps - a.steps // 10
    print(f"{a.steps} steps of {a.batch} sequences, {q_heads}/{kv_heads} heads of {dim}: "
          f"{begin.elapsed_time(end) / n * 1e3:.1f} us a step, {block.length} slots held of {block.tokens} tokens seen")


if __name__ == "__main__":
    main()
