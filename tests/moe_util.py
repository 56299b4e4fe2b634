"""Helpers of the expert-layer tests: routed slots, and the operators'
definitions in 64 bits (plain torch, no code shared with the library)."""
from __future__ import annotations

import torch

DEV = "cuda:0"
DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "e4m3": torch.float8_e4m3fn, "f32": torch.float32}
# one rounding is off by at most half a step relative to the value; below the smallest normal by half the smallest subnormal
HALF = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11, "f32": 2.0 ** -24}
TINY = {"bf16": 2.0 ** -134, "f16": 2.0 ** -25, "f32": 2.0 ** -150}
U = 2.0 ** -24        # one f32 rounding


def ids_of(qg):
    return {"f32": qg.QG_F32, "bf16": qg.QG_BF16, "f16": qg.QG_F16, "e4m3": qg.QG_E4M3}


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def blocks(n):
    return -(-n // 128)


def routing(tokens, k, experts, seed, away=0.0):
    """ids [tokens][k] (CPU list), unequal experts, a share of the slots without an expert here."""
    g = torch.Generator().manual_seed(seed)
    like = torch.randn(experts, generator=g)
    ids = torch.topk(torch.randn(tokens, experts, generator=g) + like, min(k, experts), 1).indices
    if k > experts:
        ids = torch.randint(0, experts, (tokens, k), generator=g)
    gone = torch.rand(tokens, k, generator=g) < away
    odd = torch.tensor([-1, experts, -2 ** 31, 2 ** 31 - 1])[torch.randint(0, 4, (tokens, k), generator=g)]
    return torch.where(gone, odd, ids).tolist()


def sorted_slots(ids, experts):
    """(offsets, order, place) by lists."""
    flat = [e for row in ids for e in row]
    groups = [[] for _ in range(experts)]
    for s, e in enumerate(flat):
        if 0 <= e < experts:
            groups[e].append(s)
    offsets, order, place = [0], [], [-1] * len(flat)
    for group in groups:
        for s in group:
            place[s] = len(order)
            order.append(s)
        offsets.append(len(order))
    return offsets, order, place


def codes_of(x):
    """The definition of 8-bit rows, block by block in 64 bits on the CPU: (codes as float8, scales f32)."""
    x = x.detach().cpu().double()
    n, width = x.shape
    codes = torch.zeros(n, width, dtype=torch.float64)
    scales = torch.zeros(n, blocks(width), dtype=torch.float64)
    for b in range(blocks(width)):
        part = x[:, 128 * b:128 * b + 128]
        top = torch.where(torch.isfinite(part), part.abs(), 0.0).amax(1)
        s = torch.full((n,), 2.0 ** -126, dtype=torch.float64)
        while bool((top > 448.0 * s).any()):
            s = torch.where(top > 448.0 * s, 2.0 * s, s)
        q = part / s[:, None]
        codes[:, 128 * b:128 * b + 128] = torch.where(torch.isfinite(q), q, float("nan"))
        scales[:, b] = s
    # |q| <= 448 and q has at most 24 significant bits, so f32 holds it (or is below half the least code)
    return codes.float().to(torch.float8_e4m3fn), scales.float()


def product(x, xs, w, ws, bounds):
    """(definition, sum of magnitudes) of the grouped product, 64 bits on x's device; w [E, O, I], ws [E, nbo, nbi] f32."""
    e_n, o, i = w.shape
    m = x.shape[0]
    y = torch.zeros(m, o, dtype=torch.float64, device=x.device)
    mag = torch.zeros_like(y)
    xd = x.double() * xs.double().repeat_interleave(128, 1)[:, :i]
    for e in range(e_n):
        a, b = bounds[e], bounds[e + 1]
        if a == b:
            continue
        s = ws[e].double().repeat_interleave(128, 0)[:o].repeat_interleave(128, 1)[:, :i]
        wd = w[e].double() * s
        y[a:b] = xd[a:b] @ wd.t()
        mag[a:b] = xd[a:b].abs() @ wd.abs().t()
    return y, mag


def guarded(shape, dtype, fill=7.0):
    """A tensor between two stretches of known bytes; check(t) says whether they are still there."""
    n = 1
    for d in shape:
        n *= d
    size = torch.empty((), dtype=dtype).element_size()
    raw = torch.full((n * size + 512,), 0xA5, dtype=torch.uint8, device=DEV)
    t = raw[256:256 + n * size].view(dtype).view(shape)
    if dtype == torch.float8_e4m3fn:
        t.view(torch.uint8).fill_(0x38)
    else:
        t.fill_(fill)
    t.guard = raw
    return t


def unharmed(t):
    return bool((t.guard[:256] == 0xA5).all()) and bool((t.guard[-256:] == 0xA5).all())
