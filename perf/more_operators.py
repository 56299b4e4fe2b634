"""The expert layer's operators on real work: routed slots sorted by expert,
token rows sent to their experts (as they are, or as 8-bit codes with a scale
for each 128 elements), experts' outputs brought back with the router's
weights, the gradient of that, and the product of 8-bit activations with 8-bit
weights that have a scale for each 128 x 128 block.

A case names one operator and its sizes.  ``prepare`` makes what a program
holds before the call, ``run`` is one call (in plain torch operations, or
through the library where ``own`` is true), ``exact`` the definition in 64
bits.  Widths are those of the library's decode and prefill workloads (5120,
7168, 16384; experts of 2048) and smaller generic ones.
"""
import math
import random

import torch

own = False

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32, "e4m3": torch.float8_e4m3fn}
BYTES = {"bf16": 2, "f16": 2, "f32": 4, "e4m3": 1}
BLOCK = 128


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def sort(name=None, **kw):
    c = dict(op="sort", tokens=1, k=8, experts=64, away=0.0)
    c.update(kw)
    return dict(c, name=name) if name else c


def dispatch(name=None, **kw):
    c = dict(op="dispatch", tokens=1, k=8, experts=64, away=0.0, width=5120, src="bf16", dst="e4m3")
    c.update(kw)
    return dict(c, name=name) if name else c


def combine(name=None, **kw):
    c = dict(op="combine", tokens=1, k=8, experts=64, away=0.0, width=5120, src="bf16", dst="bf16", sorted=True)
    c.update(kw)
    return dict(c, name=name) if name else c


def grad(name=None, **kw):
    c = dict(op="grad", tokens=1, k=8, experts=64, away=0.0, width=5120, src="bf16", dst="bf16")
    c.update(kw)
    return dict(c, name=name) if name else c


def product(name=None, **kw):
    c = dict(op="product", rows=8, experts=64, used=8, inner=7168, outer=2048, power=False, dst="bf16")
    c.update(kw)
    return dict(c, name=name) if name else c


def listed():
    return [
        # a decode step's router: all latency
        sort("sort_step", tokens=8, experts=128),
        # a long prompt, one slot in ten routed to experts that live elsewhere
        sort("sort_prompt", tokens=16384, experts=256, away=0.1),
        # a small model's batch, rows copied as they are, an odd width
        dispatch("dispatch_copy_odd", tokens=37, k=6, experts=16, width=1999, src="f16", dst="f16"),
        # a prompt's rows as codes for the 8-bit experts
        dispatch("dispatch_prompt_e4m3", tokens=4096, width=7168),
        # one token's eight experts, as the routed decode product leaves them: slot by slot, in f32
        combine("combine_one", tokens=1, width=7168, src="f32", sorted=False),
        # a prompt's expert outputs back in token order
        combine("combine_prompt", tokens=4096, width=7168, away=0.05),
        # a small layer trained in f32, an odd width
        grad("grad_small_f32", tokens=333, k=3, experts=8, width=1001, src="f32", dst="f32"),
        # a training batch
        grad("grad_batch", tokens=4096),
        # one token: eight experts' weights read for one row each
        product("product_one", rows=8, used=8, experts=64, dst="f32"),
        # a decode batch: few rows an expert, unequal, some experts without any
        product("product_batch", rows=384, used=59, inner=2048, outer=7168),
        # a prompt over all experts
        product("product_prompt", rows=24571, used=48, experts=48, inner=5120, outer=2048, power=True),
        # a prompt's 512 tokens through one large matrix
        product("product_dense", rows=512, used=1, experts=1, inner=16384, outer=7168),
    ]


def log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(max(lo, hi))))))


def draw(rng):
    op = rng.choice(["sort", "dispatch", "combine", "grad", "product", "product"])
    if op == "product":
        experts = rng.choice([1, 1, 8, 16, 32, 64])
        rows = log_int(rng, 1, 24000)
        used = min(experts, rows, log_int(rng, 1, experts))
        inner, outer = 16 * log_int(rng, 8, 1024), log_int(rng, 64, 16384)
        # no dearer than the largest listed one
        while rows * inner * outer > 24571 * 5120 * 2048 or experts * inner * outer > 64 * 7168 * 2048:
            inner, outer = max(16, inner // 32 * 16), max(1, outer // 2)
        return product(rows=rows, experts=experts, used=used, inner=inner, outer=outer, power=rng.random() < 0.5,
                       dst=rng.choice(["bf16", "bf16", "f16", "f32"]))
    experts = rng.choice([4, 8, 20, 64, 128, 256])
    k = rng.randint(1, min(8, experts))
    away = rng.choice([0.0, 0.0, 0.1, 0.9])
    if op == "sort":
        return sort(tokens=log_int(rng, 1, 131072 // k), k=k, experts=experts, away=away)
    width = log_int(rng, 64, 7168)
    if rng.random() < 0.6:
        width = (width + 15) // 16 * 16
    tokens = log_int(rng, 1, min(30000, 4096 * 8 * 5120 // (k * width)))
    a, b = rng.choice(["bf16", "bf16", "f16", "f32"]), rng.choice(["bf16", "bf16", "f16", "f32"])
    if op == "dispatch":
        return dispatch(tokens=tokens, k=k, experts=experts, away=away, width=width, src=a,
                        dst=rng.choice([a, "e4m3", "e4m3"]))
    if op == "combine":
        return combine(tokens=tokens, k=k, experts=experts, away=away, width=width, src=a, dst=b,
                       sorted=rng.random() < 0.8)
    return grad(tokens=tokens, k=k, experts=experts, away=away, width=width, src=a, dst=b)


def here(c):
    """Slots whose expert is here: a fixed number, so that the work is known."""
    slots = c["tokens"] * c["k"]
    return slots - int(slots * c["away"])


def blocks(n):
    return -(-n // BLOCK)


def work(c):
    if c["op"] == "product":
        n, i, o = c["rows"], c["inner"], c["outer"]
        scale = 1 if c["power"] else 4
        return {"bytes": n * (i + 4 * blocks(i)) + c["used"] * (o * i + scale * blocks(o) * blocks(i)) +
                n * o * BYTES[c["dst"]], "flops": 2 * n * i * o}
    slots, n = c["tokens"] * c["k"], here(c)
    if c["op"] == "sort":
        return {"bytes": 4 * slots + 4 * slots + 4 * n + 4 * (c["experts"] + 1), "flops": slots}
    w = c["width"]
    if c["op"] == "dispatch":
        codes = c["dst"] == "e4m3"
        return {"bytes": c["tokens"] * w * BYTES[c["src"]] + 4 * slots + n * w * BYTES[c["dst"]] +
                (4 * n * blocks(w) if codes else 0), "flops": 2 * c["tokens"] * w if codes else 0}
    if c["op"] == "combine":
        return {"bytes": n * w * BYTES[c["src"]] + (8 if c["sorted"] else 4) * slots +
                c["tokens"] * w * BYTES[c["dst"]], "flops": 2 * n * w}
    # reads the outputs' gradient (type dst) and the experts' rows (type src), writes the rows' gradient
    return {"bytes": c["tokens"] * w * BYTES[c["dst"]] + 2 * n * w * BYTES[c["src"]] + 12 * slots, "flops": 3 * n * w}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def generator(seed):
    return torch.Generator(device=DEV).manual_seed(seed * 1000003 + 29)


def normal(g, shape, dtype, scale=1.0):
    """Normal values, made a slice at a time (the experts' weights are large)."""
    out = torch.empty(shape, dtype=dtype, device=DEV)
    flat = out.view(-1)
    step = 1 << 26
    for at in range(0, flat.numel(), step):
        n = min(step, flat.numel() - at)
        flat[at:at + n] = (torch.randn(n, generator=g, device=DEV, dtype=torch.float32) * scale).to(dtype)
    return out


def routes(g, c):
    """What a router hands over: ids [tokens, k], distinct for a token, popular experts and others, and
    its weights.  Slots of experts that live elsewhere carry -1."""
    t, k, e = c["tokens"], c["k"], c["experts"]
    liking = torch.randn(e, generator=g, device=DEV)
    score = torch.randn(t, e, generator=g, device=DEV) + 0.7 * liking
    top = torch.topk(score, k, dim=1)
    weights = torch.softmax(top.values, 1)
    ids = top.indices.to(torch.int32)
    gone = t * k - here(c)
    if gone:
        ids.view(-1)[torch.randperm(t * k, generator=g, device=DEV)[:gone]] = -1
    return ids.contiguous(), weights.contiguous()


def activations(g, shape, dtype):
    """Hidden states: normal, a few channels much larger than the others."""
    x = torch.randn(shape, generator=g, device=DEV)
    x *= torch.where(torch.rand(shape[-1], generator=g, device=DEV) < 0.01, 30.0, 1.0)
    return x.to(dtype)


def group_rows(seed, rows, experts, used):
    """Rows of each expert: `used` experts share them, each at least one, in unequal shares."""
    r = random.Random(seed * 7 + 5)
    some = r.sample(range(experts), used)
    share = [math.exp(0.8 * r.gauss(0, 1)) for _ in some]
    total, left = sum(share), rows - used
    count = [0] * experts
    for e, s in zip(some, share):
        count[e] = 1 + int(left * s / total)
    for n in range(rows - sum(count)):
        count[some[n % used]] += 1
    return count


def prepare(c, seed):
    g = generator(seed)
    st = {"case": dict(c)}
    if c["op"] == "product":
        n, e, i, o = c["rows"], c["experts"], c["inner"], c["outer"]
        st["bounds"] = [0]
        for m in group_rows(seed, n, e, c["used"]):
            st["bounds"].append(st["bounds"][-1] + m)
        st["offsets"] = torch.tensor(st["bounds"], dtype=torch.int32, device=DEV)
        # codes of blocks whose largest value fills the type's range, as a quantiser leaves them
        st["x"] = normal(g, (n, i), TYPES["e4m3"], 100.0)
        st["x_scale"] = torch.exp2(torch.randint(-9, -5, (n, blocks(i)), generator=g, device=DEV).float())
        st["w"] = normal(g, (e, o, i), TYPES["e4m3"], 100.0)
        if c["power"]:
            st["w_scale"] = torch.randint(112, 118, (e, blocks(o), blocks(i)), generator=g, device=DEV,
                                          dtype=torch.uint8)
        else:
            st["w_scale"] = torch.exp(math.log(1e-4) + math.log(10.0) *
                                      torch.rand(e, blocks(o), blocks(i), generator=g, device=DEV))
        st["y"] = torch.zeros(n, o, dtype=TYPES[c["dst"]], device=DEV)
    else:
        st["ids"], st["weights"] = routes(g, c)
        slots = c["tokens"] * c["k"]
        if c["op"] == "sort":
            st["offsets"] = torch.zeros(c["experts"] + 1, dtype=torch.int32, device=DEV)
            st["order"] = torch.full((slots,), -1, dtype=torch.int32, device=DEV)
            st["place"] = torch.zeros(c["tokens"], c["k"], dtype=torch.int32, device=DEV)
        else:
            n = here(c)
            st["place"] = places(st["ids"], c["experts"])[2].to(torch.int32)
            w = c["width"]
            if c["op"] == "dispatch":
                st["x"] = activations(g, (c["tokens"], w), TYPES[c["src"]])
                st["rows"] = torch.zeros(n, w, dtype=TYPES[c["dst"]], device=DEV)
                st["scale"] = torch.zeros(n, blocks(w), device=DEV) if c["dst"] == "e4m3" else None
            else:
                sorted_ = c["op"] == "grad" or c["sorted"]
                st["y"] = normal(g, (n if sorted_ else slots, w), TYPES[c["src"]])
                if not sorted_:
                    # slot by slot: a slot of another place's expert has a row that nobody wrote
                    st["place"] = None if not c["away"] else torch.where(
                        st["ids"] >= 0, torch.arange(slots, device=DEV, dtype=torch.int32).view(st["ids"].shape), -1)
                st["out"] = torch.zeros(c["tokens"], w, dtype=TYPES[c["dst"]], device=DEV)
                if c["op"] == "grad":
                    st["dout"] = normal(g, (c["tokens"], w), TYPES[c["dst"]])
                    st["dy"] = torch.zeros_like(st["y"])
                    st["dweights"] = torch.zeros(c["tokens"], c["k"], device=DEV)
    if own:
        import weight_only_quantized_i4g_gb300 as qg
        st["qg"] = qg
        if c["op"] == "product":
            m = qg.qgemm_e4m3_workspace_bytes(c["rows"], c["inner"], c["outer"], c["experts"])
        elif c["op"] == "sort":
            m = qg.qg_moe_sort_workspace_bytes(c["tokens"], c["k"], c["experts"])
        else:
            m = 0
        st["ws"], st["ws_bytes"] = torch.empty(max(m, 1), dtype=torch.uint8, device=DEV), m
    return st


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

def run(st):
    return (run_own if own else run_plain)(st)


def outputs(st):
    op = st["case"]["op"]
    names = {"sort": ("offsets", "order", "place"), "dispatch": ("rows", "scale"), "combine": ("out",),
             "grad": ("dy", "dweights"), "product": ("y",)}[op]
    return {n: st[n] for n in names if st[n] is not None}


def run_own(st):
    qg, c = st["qg"], st["case"]
    ids = {"f32": qg.QG_F32, "bf16": qg.QG_BF16, "f16": qg.QG_F16, "e4m3": qg.QG_E4M3}
    if c["op"] == "product":
        fmt = qg.QG_FMT_FP8UE8M0 if c["power"] else qg.QG_FMT_FP8B128
        if c["experts"] == 1:
            qg.check(qg.qgemm_e4m3(fmt, st["y"], ids[c["dst"]], st["x"], st["x_scale"], st["w"], st["w_scale"],
                                   c["rows"], c["inner"], c["outer"], st["ws"], st["ws_bytes"]))
        else:
            qg.check(qg.qgemm_e4m3_moe(fmt, st["y"], ids[c["dst"]], st["x"], st["x_scale"], st["w"], st["w_scale"],
                                       st["offsets"], c["experts"], c["rows"], c["inner"], c["outer"], st["ws"],
                                       st["ws_bytes"]))
    elif c["op"] == "sort":
        qg.check(qg.qg_moe_sort(st["offsets"], st["order"], st["place"], st["ids"], c["tokens"], c["k"], c["experts"],
                                st["ws"], st["ws_bytes"]))
    elif c["op"] == "dispatch":
        qg.check(qg.qg_moe_dispatch(st["rows"], ids[c["dst"]], st["scale"], st["x"], ids[c["src"]], c["width"],
                                    st["place"], c["tokens"], c["k"], c["width"], st["rows"].shape[0]))
    elif c["op"] == "combine":
        qg.check(qg.qg_moe_combine(st["out"], ids[c["dst"]], st["y"], ids[c["src"]], st["weights"], st["place"],
                                   c["tokens"], c["k"], c["width"], st["y"].shape[0]))
    else:
        qg.check(qg.qg_moe_combine_grad(st["dy"], st["dweights"], st["dout"], ids[c["dst"]], st["y"], ids[c["src"]],
                                        st["weights"], st["place"], c["tokens"], c["k"], c["width"],
                                        st["y"].shape[0]))
    return outputs(st)


def run_plain(st):
    {"sort": plain_sort, "dispatch": plain_dispatch, "combine": plain_combine, "grad": plain_grad,
     "product": plain_product}[st["case"]["op"]](st)
    return outputs(st)


def places(ids, experts):
    """Offsets of the experts' rows, the slots in order, and each slot's row (-1: none).  Slots of no expert
    here sort behind the others."""
    flat = ids.reshape(-1).long()
    kept = (flat >= 0) & (flat < experts)
    by = torch.where(kept, flat, experts)
    order = torch.argsort(by, stable=True)
    count = torch.zeros(experts + 1, dtype=torch.long, device=ids.device).scatter_add_(0, by, torch.ones_like(by))
    offsets = torch.cat([torch.zeros_like(count[:1]), count[:experts].cumsum(0)])
    at = torch.empty_like(order).scatter_(0, order, torch.arange(order.numel(), device=ids.device))
    return offsets, order, torch.where(kept, at, -1).view(ids.shape)


def plain_sort(st):
    offsets, order, place = places(st["ids"], st["case"]["experts"])
    st["offsets"].copy_(offsets)
    n = here(st["case"])
    st["order"][:n] = order[:n]
    st["place"].copy_(place)


def power_scale(top):
    """2^e with the least e >= -126 for which top <= 448 * 2^e (448 = 0.875 * 2^9: the type's largest)."""
    m, e = torch.frexp(top)
    e = torch.where(m > 0.875, e - 8, e - 9).clamp_min(-126)
    e = torch.where(top == 0, -126, e)
    return ((e + 127).to(torch.int32) << 23).view(torch.float32)


def plain_dispatch(st):
    c = st["case"]
    place, x = st["place"], st["x"]
    t, j = (place >= 0).nonzero(as_tuple=True)
    at = place[t, j].long()
    if c["dst"] != "e4m3":
        st["rows"][at] = x[t]
        return
    w = c["width"]
    x = torch.nn.functional.pad(x.float(), (0, blocks(w) * BLOCK - w)).view(c["tokens"], -1, BLOCK)
    scale = power_scale(torch.where(torch.isfinite(x), x.abs(), 0.0).amax(-1))
    codes = (x / scale[..., None]).to(TYPES["e4m3"]).view(torch.uint8).view(c["tokens"], -1)[:, :w]
    st["rows"].view(torch.uint8)[at] = codes[t]         # torch writes 8-bit floats through a view of their bits
    st["scale"][at] = scale[t]


def placed(st):
    """Each slot's row of y in f32, zero for a slot without one: [tokens, k, width]."""
    c, y, place = st["case"], st["y"], st["place"]
    if place is None:
        return y.float().view(c["tokens"], c["k"], -1), None
    rows = y[place.clamp_min(0).long()].float()
    return rows.masked_fill_((place < 0)[..., None], 0.0), place


def plain_combine(st):
    rows, _ = placed(st)
    st["out"].copy_((rows * st["weights"][..., None]).sum(1))


def plain_grad(st):
    rows, place = placed(st)
    d = st["dout"].float()
    st["dweights"].copy_((rows * d[:, None]).sum(-1))
    del rows
    t, j = (place >= 0).nonzero(as_tuple=True)
    st["dy"][place[t, j].long()] = (st["weights"][t, j][:, None] * d[t]).to(st["dy"].dtype)


def plain_product(st):
    c = st["case"]
    i, o = c["inner"], c["outer"]
    ws = st["w_scale"]
    if c["power"]:
        ws = torch.where(ws == 0, 2.0 ** -127, (ws.to(torch.int32) << 23).view(torch.float32))
    for e in range(c["experts"]):
        a, b = st["bounds"][e], st["bounds"][e + 1]
        if a == b:
            continue
        x = st["x"][a:b].float() * st["x_scale"][a:b].repeat_interleave(BLOCK, 1)[:, :i]
        s = ws[e].repeat_interleave(BLOCK, 0)[:o].repeat_interleave(BLOCK, 1)[:, :i]
        st["y"][a:b] = torch.matmul(x, (st["w"][e].float() * s).t()).to(st["y"].dtype)


# ---------------------------------------------------------------------------
# the definition in 64 bits
# ---------------------------------------------------------------------------

def exact(c, seed):
    global own
    was, own = own, False
    try:
        st = prepare(c, seed)
    finally:
        own = was
    if c["op"] == "sort":
        return exact_sort(c, st["ids"].cpu().view(-1).tolist())
    if c["op"] == "product":
        return {"y": exact_product(c, st)}
    n, w = here(c), c["width"]
    place = list(range(c["tokens"] * c["k"])) if st["place"] is None else st["place"].view(-1).tolist()
    slots = torch.tensor([s for s, p in enumerate(place) if p >= 0], device=DEV)
    rows = torch.tensor([p for p in place if p >= 0], device=DEV)
    token = slots // c["k"]
    if c["op"] == "dispatch":
        codes = torch.zeros(n, w, dtype=torch.float64, device=DEV)
        x = st["x"].double()
        if c["dst"] != "e4m3":
            codes[rows] = x[token]
            return {"rows": codes}
        scale = torch.empty(c["tokens"], blocks(w), dtype=torch.float64, device=DEV)
        for b in range(blocks(w)):
            top = x[:, b * BLOCK:(b + 1) * BLOCK].abs().amax(1)
            least = torch.full_like(top, 2.0 ** -126)
            for e in range(-125, 121):                  # the least power of two that holds the block
                least = torch.where(top > 448.0 * least, 2.0 ** e, least)
            scale[:, b] = least
            x[:, b * BLOCK:(b + 1) * BLOCK] /= least[:, None]
        codes[rows] = x[token]
        out = torch.zeros(n, blocks(w), dtype=torch.float64, device=DEV)
        out[rows] = scale[token]
        return {"rows": codes, "scale": out}
    weight = st["weights"].double().view(-1)[slots]
    if c["op"] == "combine":
        out = torch.zeros(c["tokens"], w, dtype=torch.float64, device=DEV)
        for j in range(c["k"]):
            at = slots % c["k"] == j                    # one slot of a token at a time
            out[token[at]] += st["y"].double()[rows[at]] * weight[at, None]
        return {"out": out}
    dy = torch.zeros(st["y"].shape, dtype=torch.float64, device=DEV)
    dw = torch.zeros(c["tokens"] * c["k"], dtype=torch.float64, device=DEV)
    for at in range(0, len(rows), 4096):
        r, t, s = rows[at:at + 4096], token[at:at + 4096], slots[at:at + 4096]
        d = st["dout"][t].double()
        dy[r] = weight[at:at + 4096, None] * d
        dw[s] = torch.einsum("ri,ri->r", st["y"][r].double(), d)
    return {"dy": dy, "dweights": dw.view(c["tokens"], c["k"])}


def exact_sort(c, ids):
    lists = [[] for _ in range(c["experts"])]
    for s, e in enumerate(ids):
        if 0 <= e < c["experts"]:
            lists[e].append(s)
    order = [s for group in lists for s in group]
    place = [-1] * len(ids)
    for p, s in enumerate(order):
        place[s] = p
    offsets = [0]
    for group in lists:
        offsets.append(offsets[-1] + len(group))
    order += [-1] * (len(ids) - len(order))
    ints = [torch.tensor(v, dtype=torch.int32, device=DEV) for v in (offsets, order, place)]
    return {"offsets": ints[0], "order": ints[1], "place": ints[2].view(c["tokens"], c["k"])}


def exact_product(c, st):
    """Block by block of 128: the codes' sums, which 64 bits hold exactly, times the two scales."""
    if c["rows"] * c["inner"] * c["outer"] > 4e11:
        return None
    n, i, o = c["rows"], c["inner"], c["outer"]
    y = torch.zeros(n, o, dtype=torch.float64, device=DEV)
    for e in range(c["experts"]):
        a, b = st["bounds"][e], st["bounds"][e + 1]
        if a == b:
            continue
        s = st["w_scale"][e].double()
        if c["power"]:
            s = 2.0 ** (s - 127.0)
        for k in range(blocks(i)):
            part = st["x"][a:b, k * BLOCK:(k + 1) * BLOCK].double() @ st["w"][e][:, k * BLOCK:(k + 1) * BLOCK].double().t()
            part *= st["x_scale"][a:b, k].double()[:, None]
            for m in range(blocks(o)):
                part[:, m * BLOCK:(m + 1) * BLOCK] *= s[m, k]
            y[a:b] += part
    return y
