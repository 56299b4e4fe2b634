"""Helpers of the attention-block tests: paged caches on the GPU and the
operators' definitions in 64 bits (plain torch, one sequence and head at a
time, no code shared with the library)."""
from __future__ import annotations

import math

import torch

DEV = "cuda:0"
DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "e4m3": torch.float8_e4m3fn, "f32": torch.float32}


def ids(qg):
    return {"f32": qg.QG_F32, "bf16": qg.QG_BF16, "f16": qg.QG_F16, "e4m3": qg.QG_E4M3}


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


class Paged:
    """A cache with a block table of shuffled pages; every slot of the pool
    holds `fill` (NaN by default) until written."""

    def __init__(self, qg, lens, heads, dim, kv="bf16", page=16, seed=0, weight=False, order="head", extra=2,
                 width=None, fill=float("nan")):
        g = torch.Generator().manual_seed(seed)
        self.qg, self.kv, self.page, self.heads, self.dim, self.order = qg, kv, page, heads, dim, order
        self.lens_list = list(lens)
        count = [-(-n // page) for n in lens]
        self.n_pages = sum(count) + extra
        perm = torch.randperm(self.n_pages, generator=g).tolist()
        self.width = width or max(max(count), 1)
        table = [[-1] * self.width for _ in lens]
        for b, n in enumerate(count):
            for i in range(n):
                table[b][i] = perm.pop()
        self.free = perm
        self.table = ints(table)
        self.lens = ints(lens)
        shape = (self.n_pages, heads, page, dim) if order == "head" else (self.n_pages, page, heads, dim)
        self.k = torch.full(shape, fill, dtype=torch.float32, device=DEV).to(DTYPES[kv])
        self.v = self.k.clone()
        self.k_scale = self.v_scale = None
        if kv == "e4m3":
            self.k_scale = (0.5 + torch.rand(heads, generator=g)).to(DEV) / 64
            self.v_scale = (0.5 + torch.rand(heads, generator=g)).to(DEV) / 64
        self.weight = torch.full((self.n_pages, heads, page), 0.25, device=DEV) if weight else None
        self.cache = qg.kv_cache(self.k, self.v, self.k_scale, self.v_scale, self.weight, order=order)
        self.gen = g

    def randn(self, *shape):
        return torch.randn(*shape, generator=self.gen).to(DEV)

    def where(self, b, n=None):
        """(pages, slots in page) of sequence b's first n slots."""
        n = self.lens_list[b] if n is None else n
        t = torch.arange(n, device=DEV)
        return self.table[b].long()[t // self.page], t % self.page

    def put(self, name, b, h, x):
        """Write x f32 [n, dim] (values, or code values for e4m3) to sequence b's first n slots."""
        pool = getattr(self, name)
        p, o = self.where(b, x.shape[0])
        x = x.to(DTYPES[self.kv])
        if self.kv == "e4m3":
            pool, x = pool.view(torch.uint8), x.view(torch.uint8)
        if self.order == "head":
            pool[p, h, o] = x
        else:
            pool[p, o, h] = x

    def get(self, name, b, h, n=None):
        """f64 [n, dim] of sequence b's slots, scales applied."""
        pool = getattr(self, name)
        p, o = self.where(b, n)
        raw = pool.view(torch.uint8) if self.kv == "e4m3" else pool
        x = raw[p, h, o] if self.order == "head" else raw[p, o, h]
        x = x.view(pool.dtype).double()
        if self.kv == "e4m3":
            x = x * getattr(self, name + "_scale")[h].double()
        return x

    def fill(self, scale=None):
        scale = scale or (40.0 if self.kv == "e4m3" else 1.0)
        for b, n in enumerate(self.lens_list):
            for h in range(self.heads):
                self.put("k", b, h, scale * self.randn(n, self.dim))
                self.put("v", b, h, scale * self.randn(n, self.dim))
        return self


def attention(pc, q, S, hq, scale):
    """Definition in 64 bits: o, lse, per-slot weights by (b, h), and the error
    scales of z (sum |q k| scale) and o (sum p |v|)."""
    B = len(pc.lens_list)
    G = hq // pc.heads
    o = torch.zeros(B, S, hq, pc.dim, dtype=torch.float64, device=DEV)
    mag_o = torch.zeros_like(o)
    lse = torch.full((B, S, hq), -math.inf, dtype=torch.float64, device=DEV)
    mag_z = torch.zeros(B, S, hq, dtype=torch.float64, device=DEV)
    w = {}
    q = q.double().view(B, S, hq, pc.dim)
    for b, n in enumerate(pc.lens_list):
        for h in range(pc.heads):
            k, v = pc.get("k", b, h), pc.get("v", b, h)
            w[b, h] = torch.zeros(n, dtype=torch.float64, device=DEV)
            for i in range(S):
                m = n - S + 1 + i
                if m <= 0:
                    continue
                hs = slice(h * G, (h + 1) * G)
                z = (q[b, i, hs] @ k[:m].T) * scale
                p = torch.softmax(z, -1)
                o[b, i, hs] = p @ v[:m]
                mag_o[b, i, hs] = p @ v[:m].abs()
                lse[b, i, hs] = torch.logsumexp(z, -1)
                mag_z[b, i, hs] = ((q[b, i, hs].abs() @ k[:m].abs().T) * abs(scale)).amax(-1)
                w[b, h][:m] += p.sum(0)
    return o, lse, w, mag_o, mag_z


# largest relative error of one rounding to p significant bits (nearest even):
# half a step of 2^(1-p), relative to a value just above a power of two: 2^-p
HALF_ULP = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8, "f16": 2.0 ** -11}


def run_attention(pc, q, S, hq, scale, out="f32", accumulate=False, lse=True, max_len=None, stream=None):
    qg = pc.qg
    B = len(pc.lens_list)
    max_len = max(pc.lens_list + [1]) if max_len is None else max_len
    o = torch.full((B * S, hq, pc.dim), float("nan"), dtype=DTYPES[out], device=DEV)
    ls = torch.full((B * S, hq), float("nan"), device=DEV) if lse else None
    n = qg.qattn_workspace_bytes(pc.cache, B, max_len, S, hq, int(accumulate))
    ws = torch.full((max(n, 1),), 255, dtype=torch.uint8, device=DEV)      # contents must not matter
    qt = "f16" if q.dtype == torch.float16 else "bf16"
    qg.check(qg.qattn_paged(pc.cache, pc.table, pc.width, pc.lens, B, max_len, o, ids(qg)[out], ls, q, ids(qg)[qt],
                            q.shape[-1] if q.dim() == 2 else q.stride(0), S, hq, scale, int(accumulate), ws, n,
                            stream))
    return o, ls


def check_attention(pc, q, S, hq, scale, out="f32", accumulate=False, **kw):
    """Runs the call and holds it to the definition.  The bounds: z sums D
    products in f32 (possibly truncating adders, so 2^-22 of sum |q k| a term),
    which moves exp(z - lse) by twice that relatively; p is held in at least 16
    bits (2^-16), sums of p in f32 add 2^-18; the output is rounded once."""
    o64, lse64, w64, mag_o, mag_z = attention(pc, q, S, hq, scale)
    before = pc.weight.clone() if accumulate else None
    o, lse = run_attention(pc, q, S, hq, scale, out, accumulate, **kw)
    torch.cuda.synchronize()
    rc, status = pc.qg.qg_device_status()
    assert rc == 0 and status == 0, status
    tz = pc.dim * 2.0 ** -22 * mag_z + 2.0 ** -20
    B = len(pc.lens_list)
    o = o.double().view(B, S, hq, pc.dim)
    bound = (2 * tz + 2.0 ** -15)[..., None] * mag_o + HALF_ULP[out] * o64.abs() + (2.0 ** -24 if out == "f16" else 0)
    err = (o - o64).abs()
    assert bool((err <= bound).all()), float((err - bound).max())
    if lse is not None:
        empty = lse64 == -math.inf
        l = lse.double().view(B, S, hq)
        assert bool((l[empty] == -math.inf).all()) and bool((o[empty] == 0).all())
        bl = (tz + 2.0 ** -22 * lse64.abs())[~empty]
        assert bool(((l - lse64).abs()[~empty] <= bl).all()), float(((l - lse64).abs()[~empty] - bl).max())
    if accumulate:
        rows = S * hq // pc.heads
        want = before.double()
        tol = torch.zeros_like(want)
        for (b, h), w in w64.items():
            p, i = pc.where(b)
            want[p, h, i] += w
            t = float((2 * tz[b]).max()) + 2.0 ** -18
            tol[p, h, i] = t * w + 2.0 ** -22 * rows
        err = (pc.weight.double() - want).abs()
        assert bool((err <= tol + 2.0 ** -23 * want.abs()).all()), float((err - tol).max())
    return o, lse
