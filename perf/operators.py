"""The attention block's operators on real work: rotary positions and the
cache write, attention of new tokens over a paged key-value cache, and
eviction from that cache by accumulated attention weight.

A case names one operator and its sizes.  ``prepare`` makes what a serving
program holds before the call, ``run`` is one call (in plain torch operations,
or through the library where ``own`` is true), ``exact`` the definition in 64
bits.  Head counts are those of hidden sizes 5120 (40 heads) and 7168 (56
heads) at 128 a head with 8 key-value heads, and smaller generic ones.
"""
import math

import torch

own = False

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "e4m3": torch.float8_e4m3fn, "f32": torch.float32}
BYTES = {"bf16": 2, "f16": 2, "e4m3": 1, "f32": 4}


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def append(name=None, **kw):
    c = dict(op="append", tokens=1, seqs=1, hq=40, hkv=8, dim=128, rotary=128, axes=1, interleaved=False, kv="bf16",
             src="f32", page=16, past=1000)
    c.update(kw)
    return dict(c, name=name) if name else c


def attn(name=None, **kw):
    c = dict(op="attn", seqs=1, lo=1, hi=1, new=1, hq=40, hkv=8, dim=128, kv="bf16", out="bf16", page=16,
             weights=False)
    c.update(kw)
    return dict(c, name=name) if name else c


def evict(name=None, **kw):
    c = dict(op="evict", seqs=1, lo=1, hi=1, budget=1, sinks=4, recent=32, hkv=8, dim=128, kv="bf16", page=16)
    c.update(kw)
    return dict(c, name=name) if name else c


def listed():
    return [
        # one sequence, one new token: the smallest call of a decode step, all latency
        append("append_one"),
        # a decode batch into an 8-bit cache, rotating half of each head
        append("append_batch_e4m3", tokens=96, seqs=96, hq=56, rotary=64, kv="e4m3", page=64, past=3001),
        # several prompts at once with time/height/width positions, as image tokens carry them
        append("append_prompt_3axis", tokens=6001, seqs=5, axes=3, past=0),
        # the first tokens of a chat: a short cache, all latency
        attn("attn_one_short", lo=130, hi=130),
        # one long document, one reader: the cache's length is all there is to split
        attn("attn_one_long", lo=131071, hi=131071, hq=56, page=32),
        # a serving batch of unequal ages, some just begun, one without a token
        attn("attn_batch_ragged", seqs=48, lo=0, hi=8190),
        # four drafted tokens a sequence, small heads, f32 out for the int4 output projection
        attn("attn_draft_f16", seqs=16, lo=3, hi=4099, new=4, hq=32, hkv=4, dim=64, kv="f16", out="f32"),
        # the largest: long contexts in an 8-bit cache
        attn("attn_e4m3_large", seqs=64, lo=6000, hi=16384, hq=56, kv="e4m3", page=64),
        # the same attention with the weights summed up for a later eviction
        attn("attn_weights", seqs=9, lo=500, hi=8192, weights=True),
        # one sequence a little over its budget
        evict("evict_one", lo=1280, hi=1280, budget=1024),
        # a batch cut to half, the shorter ones left whole
        evict("evict_batch", seqs=24, lo=1500, hi=8191, budget=4096, recent=256),
        # long 8-bit caches cut to a third
        evict("evict_long_e4m3", seqs=3, lo=90001, hi=100003, budget=32768, recent=1024, kv="e4m3", page=64),
    ]


def log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "attn", "attn", "evict"])
    kv = rng.choice(["bf16", "bf16", "f16", "e4m3"])
    hkv = rng.choice([1, 2, 4, 5, 8])
    dim = rng.choice([64, 80, 128, 128, 256])
    page = rng.choice([16, 16, 24, 32, 64, 128])
    hq = hkv * rng.randint(1, 8)
    if op == "append":
        seqs = log_int(rng, 1, 64)
        return append(tokens=max(seqs, log_int(rng, 1, 6000)), seqs=seqs, hq=hq, hkv=hkv, dim=dim,
                      rotary=rng.choice([dim, dim // 2]), axes=rng.choice([1, 1, 2, 3]),
                      interleaved=rng.random() < 0.4, kv=kv, src=rng.choice(["f32", "f32", "bf16"]), page=page,
                      past=rng.choice([0, rng.randint(1, 8000)]))
    seqs = log_int(rng, 1, 48)
    new = rng.choice([1, 1, 1, 2, 3, 5, 8]) if op == "attn" else 1
    most = min(100000, int(1.4e9 / (seqs * hkv * dim * 2 * BYTES[kv])), int(2e10 / (seqs * hq * dim * 4 * new)))
    hi = log_int(rng, 40, most)
    lo = min(hi, rng.choice([0, 1, hi // 3, hi]))
    if op == "attn":
        return attn(seqs=seqs, lo=lo, hi=hi, new=new, hq=hq, hkv=hkv, dim=dim, kv=kv,
                    out=rng.choice(["f32", "bf16" if kv != "f16" else "f16"]), page=page, weights=rng.random() < 0.3)
    budget = max(1, log_int(rng, max(1, hi // 8), hi))
    sinks = rng.randint(0, min(8, budget))
    return evict(seqs=seqs, lo=lo, hi=hi, budget=budget, sinks=sinks, recent=rng.randint(0, (budget - sinks) // 2),
                 hkv=hkv, dim=dim, kv=kv, page=page)


def spread(lo, hi, n):
    """n lengths over [lo, hi], both ends among them, in no order."""
    if n == 1:
        return [hi]
    return [lo + (hi - lo) * ((i * 7919) % n) // (n - 1) if n % 7919 else hi for i in range(n)]


def q_type(c):
    return "f16" if c["kv"] == "f16" else "bf16"


def work(c):
    hkv, d, e = c["hkv"], c["dim"], BYTES[c["kv"]]
    if c["op"] == "append":
        heads = c["hq"] + 2 * hkv
        t = c["tokens"]
        return {"bytes": t * d * (heads * BYTES[c["src"]] + c["hq"] * 2 + 2 * hkv * e) + t * hkv * 4 +
                t * (8 + 4 * c["axes"]), "flops": 6 * t * (c["hq"] + hkv) * c["rotary"] // 2}
    lens = spread(c["lo"], c["hi"], c["seqs"])
    if c["op"] == "attn":
        n, s = sum(lens), c["new"]
        rows = c["seqs"] * s * c["hq"]
        return {"bytes": n * hkv * d * e * 2 + rows * (d * (2 + BYTES[c["out"]]) + 4) + 4 * len(lens) +
                4 * sum(-(-x // c["page"]) for x in lens) + (8 * n * hkv if c["weights"] else 0),
                "flops": 4 * n * s * c["hq"] * d}
    kept = sum(min(x, c["budget"]) for x in lens)
    return {"bytes": hkv * (4 * sum(lens) + kept * (4 * d * e + 12)), "flops": hkv * sum(lens)}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def generator(seed):
    return torch.Generator(device=DEV).manual_seed(seed * 1000003 + 17)


def normal(g, shape, dtype, scale=1.0):
    """Normal values, made a slice at a time (the caches are large)."""
    out = torch.empty(shape, dtype=dtype, device=DEV)
    flat = out.view(-1)
    step = 1 << 26
    for at in range(0, flat.numel(), step):
        n = min(step, flat.numel() - at)
        flat[at:at + n] = (torch.randn(n, generator=g, device=DEV, dtype=torch.float32) * scale).to(dtype)
    return out


def tables(g, counts, first, total):
    """A block table [seqs][most pages] of distinct pages in no order, taken from [first, total)."""
    width = max(max(counts), 1)
    ids = (torch.randperm(total - first, generator=g, device=DEV) + first).to(torch.int32)
    table = torch.full((len(counts), width), -1, dtype=torch.int32, device=DEV)
    at = 0
    for b, n in enumerate(counts):
        table[b, :n] = ids[at:at + n]
        at += n
    return table


def pages(lens, page):
    return [-(-x // page) for x in lens]


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def scales(g, c):
    """Per-head scales of an 8-bit cache, calibrated so that values of a few sigma stay in range."""
    if c["kv"] != "e4m3":
        return None, None
    return tuple(0.01 + 0.02 * torch.rand(c["hkv"], generator=g, device=DEV) for _ in range(2))


def prepare(c, seed):
    g = generator(seed)
    kv, hkv, d, page = TYPES[c["kv"]], c["hkv"], c["dim"], c["page"]
    st = {"case": dict(c)}
    if c["op"] == "append":
        t, n = c["tokens"], c["seqs"]
        per = [t // n + (1 if b < t % n else 0) for b in range(n)]
        past = [c["past"] if b % 3 else c["past"] // 2 for b in range(n)]
        lens = [a + b for a, b in zip(per, past)]
        count = pages(lens, page)
        total = sum(count) + 1
        st["seq"] = ints([b for b in range(n) for _ in range(per[b])])
        st["slot"] = ints([past[b] + i for b in range(n) for i in range(per[b])])
        order = st["slot"].view(-1, 1)
        # further axes: rows and columns of a picture of 32 by 32 patches
        st["pos"] = torch.cat([order, order // 32 % 32, order % 32], 1)[:, :c["axes"]].contiguous()
        half = c["rotary"] // 2
        st["axis"] = bytes(j * c["axes"] // half for j in range(half))
        j = torch.arange(half, device=DEV, dtype=torch.float64)
        st["inv_freq"] = (10000.0 ** (-2 * j / c["rotary"])).float()
        st["qkv"] = normal(g, (t, (c["hq"] + 2 * hkv) * d), TYPES[c["src"]])
        st["q"] = torch.zeros(t, c["hq"] * d, dtype=TYPES[q_type(c)], device=DEV)
        st["k"] = torch.zeros(total, hkv, page, d, dtype=kv, device=DEV)
        st["v"] = torch.zeros_like(st["k"])
        st["weight"] = normal(g, (total, hkv, page), torch.float32).abs_()
        st["table"] = tables(g, count, 0, total)
        st["k_scale"], st["v_scale"] = scales(g, c)
    else:
        lens = spread(c["lo"], c["hi"], c["seqs"])
        count = pages(lens, page)
        src = sum(count) + 1
        dst = pages([min(x, c["budget"]) for x in lens], page) if c["op"] == "evict" else [0]
        total = src + sum(dst)
        st["lens"] = ints(lens)
        st["table"] = tables(g, count, 0, src)
        st["k_scale"], st["v_scale"] = scales(g, c)
        spreadout = 50.0 if c["kv"] == "e4m3" else 1.0        # codes of a calibrated cache fill their range
        st["k"] = normal(g, (total, hkv, page, d), kv, spreadout)
        st["v"] = normal(g, (total, hkv, page, d), kv, spreadout)
        if c["op"] == "attn":
            rows = c["seqs"] * c["new"]
            st["q"] = normal(g, (rows, c["hq"] * d), TYPES[q_type(c)], 1.5)
            st["o"] = torch.zeros(rows, c["hq"] * d, dtype=TYPES[c["out"]], device=DEV)
            st["lse"] = torch.zeros(rows, c["hq"], dtype=torch.float32, device=DEV)
            st["scale"] = d ** -0.5
            st["weight"] = normal(g, (total, hkv, page), torch.float32).abs_() if c["weights"] else None
        else:
            st["first"] = src
            st["dst_table"] = tables(g, dst, src, total)
            for name in ("k", "v"):
                st[name][src:] = 0
            # sums of attention weights: a few large, many small, equal ones, and zeros of tokens nobody looked at
            w = torch.exp(1.5 * normal(g, (total, hkv, page), torch.float32))
            w = torch.where(w < 0.25, (w * 64).floor() / 64, w)
            w[src:] = 0
            st["weight"] = w
            st["kept"] = torch.zeros(c["seqs"], hkv, c["budget"], dtype=torch.int32, device=DEV)
            st["new_lens"] = torch.zeros(c["seqs"], dtype=torch.int32, device=DEV)
    if own:
        import weight_only_quantized_i4g_gb300 as qg
        st["qg"] = qg
        st["cache"] = qg.kv_cache(st["k"], st["v"], k_scale=st["k_scale"], v_scale=st["v_scale"],
                                  weight=st["weight"])
        if c["op"] == "attn":
            n = qg.qattn_workspace_bytes(st["cache"], c["seqs"], c["hi"], c["new"], c["hq"], int(c["weights"]))
            st["ws"], st["ws_bytes"] = torch.empty(max(n, 1), dtype=torch.uint8, device=DEV), n
    return st


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

def run(st):
    return (run_own if own else run_plain)(st)


def run_own(st):
    qg, c = st["qg"], st["case"]
    ids = {"f32": qg.QG_F32, "bf16": qg.QG_BF16, "f16": qg.QG_F16}
    if c["op"] == "append":
        qg.check(qg.qg_rope_append(
            st["cache"], st["table"], st["table"].shape[1], c["seqs"], st["seq"], st["slot"], c["tokens"], st["q"],
            ids[q_type(c)], st["qkv"], ids[c["src"]], st["qkv"].shape[1], c["hq"], st["pos"], c["axes"], st["axis"],
            st["inv_freq"], c["rotary"], qg.QG_ROPE_INTERLEAVED if c["interleaved"] else qg.QG_ROPE_HALF))
        return {"q": st["q"], "k": st["k"], "v": st["v"], "weight": st["weight"]}
    if c["op"] == "attn":
        qg.check(qg.qattn_paged(
            st["cache"], st["table"], st["table"].shape[1], st["lens"], c["seqs"], c["hi"], st["o"], ids[c["out"]],
            st["lse"], st["q"], ids[q_type(c)], st["q"].shape[1], c["new"], c["hq"], st["scale"], int(c["weights"]),
            st["ws"], st["ws_bytes"]))
        return attn_outputs(st)
    qg.check(qg.qg_kv_evict(
        st["cache"], st["table"], st["table"].shape[1], st["dst_table"], st["dst_table"].shape[1], st["lens"],
        c["seqs"], c["hi"], c["budget"], c["sinks"], c["recent"], st["kept"], st["new_lens"]))
    return evict_outputs(st)


def attn_outputs(st):
    out = {"o": st["o"], "lse": st["lse"]}
    if st["case"]["weights"]:
        out["weight"] = st["weight"]
    return out


def evict_outputs(st):
    at = st["first"]
    return {"kept": st["kept"], "new_lens": st["new_lens"], "k": st["k"][at:], "v": st["v"][at:],
            "weight": st["weight"][at:]}


def run_plain(st):
    return {"append": plain_append, "attn": plain_attn, "evict": plain_evict}[st["case"]["op"]](st)


def to_cache(x, scale, dtype):
    """f32 [.., heads, dim] in the cache's type; 8 bits: codes of x / scale, largest finite where it is larger."""
    if scale is None:
        return x.to(dtype)
    return (x / scale[:, None]).clamp(-448.0, 448.0).to(dtype)


def rotate(x, cos, sin, rotary, interleaved):
    """x f32 [tokens, heads, dim]; cos, sin [tokens, rotary/2]."""
    half = rotary // 2
    a, b = (x[..., 0:rotary:2], x[..., 1:rotary:2]) if interleaved else (x[..., :half], x[..., half:rotary])
    cos, sin = cos[:, None], sin[:, None]
    p, q = a * cos - b * sin, b * cos + a * sin
    turned = torch.stack([p, q], -1).flatten(-2) if interleaved else torch.cat([p, q], -1)
    return torch.cat([turned, x[..., rotary:]], -1)


def plain_append(st):
    c = st["case"]
    hq, hkv, d, page = c["hq"], c["hkv"], c["dim"], c["page"]
    x = st["qkv"].float().view(-1, hq + 2 * hkv, d)
    axis = torch.tensor(list(st["axis"]), device=x.device)
    angle = st["pos"][:, axis].float() * st["inv_freq"]
    cos, sin = angle.cos(), angle.sin()
    q = rotate(x[:, :hq], cos, sin, c["rotary"], c["interleaved"])
    k = rotate(x[:, hq:hq + hkv], cos, sin, c["rotary"], c["interleaved"])
    slot = st["slot"].long()
    at = st["table"][st["seq"].long(), slot // page].long()
    st["q"].copy_(q.reshape(st["q"].shape))
    dtype = st["k"].dtype
    if c["kv"] == "e4m3":       # torch writes 8-bit floats through a view of their bits
        st["k"].view(torch.uint8)[at, :, slot % page] = to_cache(k, st["k_scale"], dtype).view(torch.uint8)
        st["v"].view(torch.uint8)[at, :, slot % page] = to_cache(x[:, hq + hkv:], st["v_scale"], dtype).view(torch.uint8)
    else:
        st["k"][at, :, slot % page] = k.to(dtype)
        st["v"][at, :, slot % page] = x[:, hq + hkv:].to(dtype)
    st["weight"][at, :, slot % page] = 0.0
    return {"q": st["q"], "k": st["k"], "v": st["v"], "weight": st["weight"]}


def dense(pool, table):
    """The pages of a pool [pages, heads, page, ..] in table order: [seqs, heads, slots, ..]."""
    x = pool[table.clamp_min(0).long()]
    return x.transpose(1, 2).flatten(2, 3)


def plain_attn(st):
    c = st["case"]
    hkv, d, s = c["hkv"], c["dim"], c["new"]
    n, rows = c["seqs"], c["hq"] // hkv * s
    bits = (lambda p: p.view(torch.uint8)) if c["kv"] == "e4m3" else (lambda p: p)
    k = dense(bits(st["k"]), st["table"])
    k = (k.view(TYPES["e4m3"]).float() * st["k_scale"][:, None, None]) if c["kv"] == "e4m3" else k.float()
    q = st["q"].float().view(n, s, hkv, -1, d).permute(0, 2, 3, 1, 4).reshape(n, hkv, rows, d)
    z = torch.matmul(q, k.transpose(2, 3)) * st["scale"]            # [n, hkv, rows, slots]
    del k
    slot = torch.arange(z.shape[-1], device=z.device)
    limit = st["lens"][:, None] - s + 1 + torch.arange(s, device=z.device)        # [n, s]
    seen = slot < limit.repeat(1, rows // s)[:, None, :, None]
    z = z.masked_fill(~seen, -math.inf)
    top = z.amax(-1, keepdim=True)
    e = torch.exp(z - top.masked_fill(top == -math.inf, 0.0))
    total = e.sum(-1, keepdim=True)
    p = e / total.masked_fill(total == 0, 1.0)
    v = dense(bits(st["v"]), st["table"])
    v = (v.view(TYPES["e4m3"]).float() * st["v_scale"][:, None, None]) if c["kv"] == "e4m3" else v.float()
    # slots past the end were read from some page all the same: they weigh nothing, whatever they hold
    v = v.masked_fill((slot >= st["lens"][:, None])[:, None, :, None], 0.0)
    o = torch.matmul(p, v)
    del v
    st["o"].copy_(o.view(n, hkv, -1, s, d).permute(0, 3, 1, 2, 4).reshape(st["o"].shape))
    lse = (top + total.log()).view(n, hkv, -1, s).permute(0, 3, 1, 2)
    st["lse"].copy_(lse.reshape(st["lse"].shape))
    if c["weights"]:
        held = (st["table"] >= 0)
        more = p.sum(2).view(n, hkv, -1, c["page"]).transpose(1, 2)          # [n, pages, hkv, page]
        st["weight"][st["table"][held].long()] += more[held]
    return attn_outputs(st)


def plain_evict(st):
    c = st["case"]
    n, hkv, page, budget = c["seqs"], c["hkv"], c["page"], c["budget"]
    w = dense(st["weight"], st["table"])                                     # [n, hkv, slots]
    slot = torch.arange(w.shape[-1], device=w.device)
    lens = st["lens"].long()[:, None, None]
    new = lens.clamp_max(budget)
    safe = (slot < c["sinks"]) | (slot >= lens - c["recent"])
    w = w.masked_fill(safe, math.inf).masked_fill(slot >= lens, -math.inf)
    if w.shape[-1] < budget:
        w = torch.nn.functional.pad(w, (0, budget - w.shape[-1]), value=-math.inf)
    best = torch.sort(w, dim=-1, descending=True, stable=True).indices[..., :budget]
    rank = torch.arange(budget, device=w.device)
    best = torch.where(rank < new, best, 1 << 30).sort(-1).values
    used = (rank < new).expand(n, hkv, budget)
    st["kept"].copy_(torch.where(used, best, -1))
    st["new_lens"].copy_(new[:, 0, 0])
    b, h, i = used.nonzero(as_tuple=True)
    at = best[b, h, i]
    src, dst = st["table"][b, at // page].long(), st["dst_table"][b, i // page].long()
    for name in ("k", "v", "weight"):
        pool = st[name].view(torch.uint8) if c["kv"] == "e4m3" and name != "weight" else st[name]
        pool[dst, h, i % page] = pool[src, h, at % page]
    return evict_outputs(st)


# ---------------------------------------------------------------------------
# the definition in 64 bits, one sequence or head at a time
# ---------------------------------------------------------------------------

def exact(c, seed):
    global own
    was, own = own, False
    try:
        st = prepare(c, seed)
    finally:
        own = was
    return {"append": exact_append, "attn": exact_attn, "evict": exact_evict}[c["op"]](c, st)


def exact_append(c, st):
    hq, hkv, d, page = c["hq"], c["hkv"], c["dim"], c["page"]
    x = st["qkv"].double().reshape(-1, hq + 2 * hkv, d)
    freq = st["inv_freq"].double()
    half = c["rotary"] // 2
    out = x.clone()
    for j in range(half):
        i0, i1 = (2 * j, 2 * j + 1) if c["interleaved"] else (j, j + half)
        a = st["pos"][:, st["axis"][j]].double() * freq[j]
        co, si = torch.cos(a)[:, None], torch.sin(a)[:, None]
        u, w = x[:, :hq + hkv, i0], x[:, :hq + hkv, i1]
        out[:, :hq + hkv, i0] = u * co - w * si
        out[:, :hq + hkv, i1] = w * co + u * si
    pools = {}
    seq, slot = st["seq"].long(), st["slot"].long()
    at = st["table"][seq, torch.div(slot, page, rounding_mode="floor")].long()
    for name, y in (("k", out[:, hq:hq + hkv]), ("v", out[:, hq + hkv:])):
        if c["kv"] == "e4m3":
            y = torch.clamp(y / st[name + "_scale"].double()[:, None], -448.0, 448.0)
        pool = st[name].double()
        pool[at, :, slot % page] = y
        pools[name] = pool
    w = st["weight"].double()
    w[at, :, slot % page] = 0.0
    return {"q": out[:, :hq].reshape(st["q"].shape), "k": pools["k"], "v": pools["v"], "weight": w}


def exact_attn(c, st):
    hkv, d, s, page = c["hkv"], c["dim"], c["new"], c["page"]
    group = c["hq"] // hkv
    lens = st["lens"].tolist()
    if sum(lens) * c["hq"] * s * d > 2e11:
        return None
    o = torch.zeros(len(lens), s, c["hq"], d, dtype=torch.float64, device=DEV)
    lse = torch.full((len(lens), s, c["hq"]), -math.inf, dtype=torch.float64, device=DEV)
    weight = st["weight"].double() if c["weights"] else None
    q = st["q"].double().reshape(len(lens), s, c["hq"], d)
    for b, n in enumerate(lens):
        if n == 0:
            continue
        ids = st["table"][b, :-(-n // page)].long()
        for h in range(hkv):
            k, v = (st[x][ids, h].double().reshape(-1, d)[:n] for x in ("k", "v"))
            if c["kv"] == "e4m3":
                k, v = k * st["k_scale"][h].double(), v * st["v_scale"][h].double()
            heads = slice(h * group, (h + 1) * group)
            for i in range(s):
                m = n - s + 1 + i
                if m <= 0:
                    continue
                z = torch.einsum("gd,td->gt", q[b, i, heads], k[:m]) * st["scale"]
                p = torch.softmax(z, -1)
                o[b, i, heads] = p @ v[:m]
                lse[b, i, heads] = torch.logsumexp(z, -1)
                if c["weights"]:
                    t = torch.arange(m, device=DEV)
                    weight[ids[t // page], h, t % page] += p.sum(0)
    out = {"o": o.reshape(st["o"].shape), "lse": lse.reshape(st["lse"].shape)}
    if c["weights"]:
        out["weight"] = weight
    return out


def exact_evict(c, st):
    hkv, page, budget, at0 = c["hkv"], c["page"], c["budget"], st["first"]
    pools = {x: st[x].to(torch.float32 if x == "weight" else st[x].dtype) for x in ("k", "v", "weight")}
    if sum(p.numel() for p in pools.values()) > 5e8:
        return None
    out = {x: p[at0:].double() for x, p in pools.items()}
    for b, n in enumerate(st["lens"].tolist()):
        for h in range(hkv):
            if n == 0:
                continue
            t = torch.arange(n, device=DEV)
            ids = st["table"][b].long()[t // page]
            w = pools["weight"][ids, h, t % page].double().cpu().tolist()
            middle = [i for i in range(n) if i >= c["sinks"] and i < n - c["recent"]]
            room = min(n, budget) - (n - len(middle))
            chosen = set(sorted(middle, key=lambda i: (-w[i], i))[:room]) if n > budget else set(middle)
            inside = set(middle)
            kept = torch.tensor([i for i in range(n) if i not in inside or i in chosen], device=DEV)
            i = torch.arange(len(kept), device=DEV)
            to = st["dst_table"][b].long()[i // page] - at0
            for x, p in pools.items():
                raw = p.view(torch.uint8) if p.dtype == TYPES["e4m3"] else p
                row = raw[ids[kept], h, kept % page]
                out[x][to, h, i % page] = (row.view(p.dtype) if raw is not p else row).double()
    # which slots were kept is compared as whole numbers already
    return {"kept": None, "new_lens": None, "k": out["k"], "v": out["v"], "weight": out["weight"]}
