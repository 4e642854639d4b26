"""The serving operators on a KV cache, as they are measured: rotary positions
(a training pass and the append of new tokens to a paged cache), attention for
a tree of drafted tokens over that cache, the attention weight that each cached
token collects, and eviction by that weight into a packed buffer.

`run` computes each in a plain form (elementary torch operations in 32 bits,
rounded once at the end) or, where `own` is true, through the package's entry
points. `exact` is the definition in 64 bits.

One layer's cache is a pool of pages [pages, kv heads, page tokens, head dim]
for K and one for V, a page table [sequences, pages of a sequence] and the
length of each sequence. The `t` new tokens of sequence b take the slots
lengths[b] .. lengths[b] + t - 1. Slots that no sequence uses hold NaN.
"""
import math
import random

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32, "e5m2": torch.float8_e5m2}
BYTES = {"bf16": 2, "fp16": 2, "fp32": 4, "e5m2": 1}


# ------------------------------------------------------------------- cases

def listed():
    return [
        # A training step's queries and keys (64 + 8 heads side by side in one projection), forward and gradient.
        dict(name="rotary train bf16", op="rotary", b=4, t=4097, heads=72, d=128, rd=128, layout="half",
             scaling="none", type="bf16"),
        # Half of each head rotated, pairs side by side, frequencies ramped for a long context; a short fp32 batch.
        dict(name="rotary part fp32", op="rotary", b=1, t=333, heads=7, d=96, rd=48, layout="interleaved",
             scaling="ramp", type="fp32"),
        # One decoding step of a batch: one new token a sequence.
        dict(name="append step bf16", op="append", b=48, t=1, n=250, hq=64, hk=8, d=128, rd=128, page=16,
             layout="half", scaling="none", type="bf16", cache="bf16"),
        # A chunk of a prompt into an FP8 cache, half of each head rotated, sequences of unequal length.
        dict(name="append chunk e5m2", op="append", b=3, t=1365, n=2000, hq=32, hk=8, d=128, rd=64, page=64,
             layout="interleaved", scaling="linear", type="fp16", cache="e5m2"),
        # One sequence, one token, a short context: latency.
        dict(name="attend one short", op="attend", b=1, t=1, n=777, hq=32, hk=8, d=128, page=16,
             type="bf16", cache="bf16"),
        # A decoding batch at long contexts of unequal length: the cache's bytes.
        dict(name="attend step bf16", op="attend", b=40, t=1, n=16384, hq=64, hk=8, d=128, page=16,
             type="bf16", cache="bf16"),
        # Small drafted trees over an FP8 cache, five query heads a KV head, pages that end inside a tile.
        dict(name="attend tree e5m2", op="attend", b=12, t=17, n=5001, hq=40, hk=8, d=64, page=48,
             type="bf16", cache="e5m2"),
        # Large drafted trees over long contexts: the products.
        dict(name="attend tree fp16", op="attend", b=2, t=64, n=65536, hq=64, hk=8, d=128, page=64,
             type="fp16", cache="fp16"),
        # The last tokens of a long prompt weigh its cache before it is evicted and sent.
        dict(name="mass window bf16", op="mass", b=1, t=32, n=131072, hq=64, hk=8, d=128, page=64,
             type="bf16", cache="bf16"),
        # A verified step of a batch adds its weights to an FP8 cache's.
        dict(name="mass step e5m2", op="mass", b=24, t=5, n=3001, hq=32, hk=8, d=64, page=16,
             type="bf16", cache="e5m2"),
        # A long prompt's cache cut to an eighth and packed to be encoded and sent.
        dict(name="evict long bf16", op="evict", b=1, n=131072, keep=16384, hk=8, d=128, page=64, cache="bf16"),
        # A batch of short FP8 caches cut to a budget, some of them already below it.
        dict(name="evict batch e5m2", op="evict", b=20, n=3001, keep=500, hk=8, d=64, page=16, cache="e5m2"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rotary", "append", "attend", "attend", "mass", "evict"])
    hk = rng.choice([1, 2, 4, 8])
    hq = hk * rng.choice([1, 2, 3, 4, 5, 8])
    d = rng.choice([64, 64, 80, 96, 128, 128, 128])
    rot = dict(rd=rng.choice([d, d // 2]), layout=rng.choice(["half", "interleaved"]),
               scaling=rng.choice(["none", "linear", "ramp"]))
    page = rng.choice([16, 16, 32, 48, 64, 128, 400])
    while True:
        if op == "rotary":
            c = dict(op=op, b=_log(rng, 1, 16), t=_log(rng, 1, 8192), heads=_log(rng, 1, 96), d=d, **rot,
                     type=rng.choice(["bf16", "fp16", "fp32"]))
        elif op == "append":
            c = dict(op=op, b=_log(rng, 1, 64), t=_log(rng, 1, 2048), n=_log(rng, 4, 2000), hq=hq, hk=hk, d=d,
                     page=page, **rot, type=rng.choice(["bf16", "fp16"]), cache="")
        elif op == "attend":
            c = dict(op=op, b=_log(rng, 1, 64), t=_log(rng, 1, 64), n=_log(rng, 16, 131072), hq=hq, hk=hk, d=d,
                     page=page, type=rng.choice(["bf16", "fp16"]), cache="")
        elif op == "mass":
            c = dict(op=op, b=_log(rng, 1, 32), t=_log(rng, 1, 64), n=_log(rng, 16, 131072), hq=hq, hk=hk, d=d,
                     page=page, type=rng.choice(["bf16", "fp16"]), cache="")
        else:
            n = _log(rng, 64, 131072)
            c = dict(op=op, b=_log(rng, 1, 32), n=n, keep=max(8, int(n * rng.uniform(0.05, 0.6))), hk=hk, d=d,
                     page=page, cache=rng.choice(["bf16", "fp16", "e5m2"]))
        if c.get("cache") == "":
            c["cache"] = rng.choice([c["type"], c["type"], "e5m2"])
        w = work(c)
        if w["bytes"] <= 1.0e9 and w["flops"] <= 2.0e11 and c["b"] * c["t"] * c["hq"] * c["n"] <= 4e8 \
                if op in ("attend", "mass") else w["bytes"] <= 1.0e9:
            return c


def _lengths(case):
    """Tokens in each sequence's cache (before the new ones) and new tokens of each sequence, from the sizes alone."""
    b, n, t = case["b"], case["n"], case.get("t", 0)
    r = random.Random(b * 1000003 + n * 101 + t)
    lens = [n] + [r.randint(n // 4, n) for _ in range(b - 1)]
    counts = [t] + [r.randint((t + 1) // 2, t) for _ in range(b - 1)]
    if b >= 4:
        lens[2] = 0  # a sequence that begins
    if b >= 8:
        counts[5] = 0  # one that drafted nothing
    return lens, counts


def work(case):
    op, d = case["op"], case["d"]
    if op == "rotary":
        x = case["b"] * case["t"] * case["heads"] * d
        return {"bytes": 4 * x * BYTES[case["type"]] + 4 * case["b"] * case["t"], "flops": 6 * x}
    lens, counts = _lengths(case)
    hk, ce = case["hk"], BYTES[case["cache"]]
    if op == "append":
        new = sum(counts)
        e = BYTES[case["type"]]
        return {"bytes": new * d * ((2 * case["hq"] + 2 * hk) * e + 2 * hk * ce + 4),
                "flops": 3 * new * d * (case["hq"] + hk)}
    if op in ("attend", "mass"):
        hq, e = case["hq"], BYTES[case["type"]]
        live = [(n + c, c) for n, c in zip(lens, counts) if c]
        keys = sum(n for n, _ in live)
        pairs = sum(n * c for n, c in live)
        rows = case["b"] * case["t"] * hq
        if op == "attend":
            return {"bytes": keys * hk * 2 * d * ce + rows * (2 * d * e + 4), "flops": 4 * pairs * hq * d}
        slots = case["b"] * hk * _capacity(case)
        return {"bytes": keys * hk * (d * ce + 4) + 4 * slots + rows * (d * e + 4), "flops": 2 * pairs * hq * d}
    kept = sum(min(n, case["keep"]) for n in lens)
    return {"bytes": 4 * hk * sum(lens) + hk * kept * 4 * d * ce + 8 * case["b"] * hk * case["keep"], "flops": hk * sum(lens)}


def _capacity(case):
    return -(-(case["n"] + case.get("t", 0)) // case["page"]) * case["page"]


# ------------------------------------------------------------------ inputs

def _freqs(case):
    """Rotation of each pair in radians a position, and the factor on both products, from the definition."""
    rd, base, scaling = case["rd"], 10000.0, case["scaling"]
    f = [base ** (-2.0 * i / rd) for i in range(rd // 2)]
    if scaling == "linear":
        return [v / 4.0 for v in f], 1.0
    if scaling == "ramp":
        turns = [4096.0 * v / (2 * math.pi) for v in f]
        mix = [min(1.0, max(0.0, (r - 1.0) / (32.0 - 1.0))) for r in turns]
        return [v * (g + (1 - g) / 8.0) for v, g in zip(f, mix)], 0.1 * math.log(8.0) + 1.0
    return f, 1.0


def _plan(case):
    import lossless_bf16_exponent_gb300 as uz

    kw = {"linear": dict(factor=4.0), "ramp": dict(factor=8.0, original_length=4096)}.get(case["scaling"], {})
    return uz.rotary_plan(case["rd"], base=10000.0, layout=case["layout"], scaling=case["scaling"], **kw)


def _rotation(case, state):
    """The pairs' rates as 64-bit fixed-point turns a position, so that a position's phase is one wrapping product."""
    f, state["magnitude"] = _freqs(case)
    turns = [int(round(v / (2 * math.pi) * 2.0 ** 64)) for v in f]
    state["turns"] = torch.tensor([v - (1 << 64) if v >= 1 << 63 else v for v in turns], device="cuda")


def _randn(g, shape, dtype, scale=None):
    x = torch.randn(shape, generator=g, device="cuda")
    return (x if scale is None else x * scale).to(dtype)


def _cache(case, g, state):
    """Pools, page table and lengths. Keys and values: per-head scales, a few strong channels."""
    lens, counts = _lengths(case)
    b, hk, d, page, t = case["b"], case["hk"], case["d"], case["page"], case.get("t", 0)
    per = _capacity(case) // page
    need = [-(-(n + t) // page) for n in lens]
    pages = sum(need) + 3
    where = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
    table = torch.full((b, per), -1, dtype=torch.int32, device="cuda")
    at = 0
    for i, m in enumerate(need):
        table[i, :m] = where[at:at + m]
        at += m
    dtype = DTYPES[case["cache"]]
    pool = torch.empty((pages, 2, hk, page, d), dtype=dtype, device="cuda")
    scale = torch.exp(math.log(0.25) + torch.rand((2, hk, 1, 1), generator=g, device="cuda") * math.log(8.0))
    gain = 1 + 3 * (torch.rand((2, hk, 1, d), generator=g, device="cuda") < 0.01).float()
    step = max(1, (1 << 26) // (2 * hk * page * d))
    for s in range(0, pages, step):
        m = min(step, pages - s)
        pool[s:s + m] = _randn(g, (m, 2, hk, page, d), dtype, scale * gain)
    used = torch.zeros((pages, page), dtype=torch.bool, device="cuda")
    n = torch.tensor(lens, device="cuda")
    upto = n if case["op"] in ("append", "evict") else n + torch.tensor(counts, device="cuda")
    slot = torch.arange(per * page, device="cuda")
    i, j = torch.nonzero(slot[None, :] < upto[:, None], as_tuple=True)
    used[table[i, j // page].long(), j % page] = True
    p, o = torch.nonzero(~used, as_tuple=True)
    raw = pool.view(torch.uint8 if dtype == torch.float8_e5m2 else torch.int16)
    raw[p, :, :, o] = 0x7F if dtype == torch.float8_e5m2 else 0x7FFF  # NaN of each type
    state.update(k=pool[:, 0], v=pool[:, 1], table=table, lengths=n.to(torch.int32),
                 counts=torch.tensor(counts, dtype=torch.int32, device="cuda"))


def _tree(case, seed):
    """Each node's ancestors and itself as bits, of a random tree for each sequence; a chain for a prompt's window."""
    r = random.Random(seed)
    b, t = case["b"], case["t"]
    chain = case["op"] == "mass"
    rows = []
    for _ in range(b):
        seen = []
        for i in range(t):
            up = i - 1 if chain else r.randint(max(-1, i - 5), i - 1) if i else -1
            seen.append((seen[up] if up >= 0 else 0) | (1 << i))
        rows.append([[v - (1 << 64) if v >= 1 << 63 else v] for v in seen])
    return torch.tensor(rows, dtype=torch.int64, device="cuda")


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    op, d = case["op"], case["d"]
    state = {"case": case}
    if op == "rotary":
        # Heads of one fused projection, whose last heads (the values) are not rotated: a strided view.
        b, t, heads = case["b"], case["t"], case["heads"]
        dtype = DTYPES[case["type"]]
        state["x"] = _randn(g, (b, t, heads + 1, d), dtype)[:, :, :heads]
        state["grad"] = _randn(g, (b, t, heads + 1, d), dtype, 1e-2)[:, :, :heads]
        first = torch.randint(0, 65536, (b, 1), generator=g, device="cuda")
        state["positions"] = (first + torch.arange(t, device="cuda")).to(torch.int32)
        _rotation(case, state)
        if own:
            state["plan"] = _plan(case)
        return state
    _cache(case, g, state)
    if op == "evict":
        # Weights collected over many steps: a few tokens hold most, many hold equal small counts.
        u = torch.rand((case["b"], case["hk"], _capacity(case)), generator=g, device="cuda")
        state["mass"] = torch.where(u < 0.2, (u * 20).floor() / 64, u.clamp_min(1e-6) ** -0.5 - 1)
        state["sink"], state["recent"] = min(4, case["keep"] // 4), case["keep"] // 4
    else:
        b, t, hq, hk = case["b"], case["t"], case["hq"], case["hk"]
        qkv = _randn(g, (b, t, hq + 2 * hk, d), DTYPES[case["type"]])
        state["q"] = qkv[:, :, :hq]
        if op == "append":
            state["knew"], state["vnew"] = qkv[:, :, hq:hq + hk], qkv[:, :, hq + hk:]
            state["positions"] = (state["lengths"][:, None] + torch.arange(t, device="cuda")).to(torch.int32)
            _rotation(case, state)
            if own:
                state["plan"] = _plan(case)
        else:
            state["mask"] = _tree(case, seed)
    if op == "mass":
        state["weights"] = (torch.rand((b, t), generator=g, device="cuda") < 0.7).float()
        state["mass"] = torch.rand((b, hk, _capacity(case)), generator=g, device="cuda") ** 4
        state["lse"] = _scores(state)[1]
    if own:
        import lossless_bf16_exponent_gb300 as uz

        state["cache"] = uz.KVCache(state["k"], state["v"], state["table"], state["lengths"])
    return state


# -------------------------------------------------------------- plain forms

def _rotated(x, positions, state, backward=False):
    case = state["case"]
    rd = case["rd"]
    phase = positions.long()[..., None] * state["turns"]  # wraps: whole turns fall away
    angle = phase.float() * (2 * math.pi / 2.0 ** 64)
    c, s = (angle.cos() * state["magnitude"])[..., None, :], (angle.sin() * state["magnitude"])[..., None, :]
    if backward:
        s = -s
    x = x.float()
    if case["layout"] == "half":
        a, b = x[..., :rd // 2], x[..., rd // 2:rd]
        y = torch.cat((a * c - b * s, b * c + a * s, x[..., rd:]), -1)
    else:
        a, b = x[..., 0:rd:2], x[..., 1:rd:2]
        y = torch.cat((torch.stack((a * c - b * s, b * c + a * s), -1).flatten(-2), x[..., rd:]), -1)
    return y


def _rows(pool, table):
    """[sequences, kv heads, capacity, head dim] of a pool, in 32 bits."""
    b, per = table.shape
    _, hk, page, d = pool.shape
    raw = pool.view(torch.uint8) if pool.dtype == torch.float8_e5m2 else pool
    x = raw[table.long()].permute(0, 2, 1, 3, 4).reshape(b, hk, per * page, d)
    return x.view(pool.dtype).float()


def _visible(state):
    """[sequences, 1, new tokens, capacity]: which cached token each new one sees; [sequences, capacity]: used slots."""
    n, c = state["lengths"].long()[:, None], state["counts"].long()[:, None]
    t = state["q"].shape[1]
    slot = torch.arange(state["table"].shape[1] * state["k"].shape[2], device="cuda")[None]
    node = slot - n  # the drafted node of a slot
    bit = (state["mask"][:, :, :1] >> node.clamp(0, 63)[:, None]) & 1
    sees = (node < 0)[:, None] | ((node >= 0) & (node < c))[:, None] & (bit != 0)
    live = torch.arange(t, device="cuda")[None] < c
    return (sees & live[..., None])[:, None], slot < n + c


def _scores(state):
    """Scaled scores [sequences, kv heads, group, new tokens, capacity] (-inf where unseen) and their log-sum-exp."""
    q, k = state["q"].float(), _rows(state["k"], state["table"])
    b, t, hq, d = q.shape
    hk = k.shape[1]
    seen, used = _visible(state)
    k = torch.where(used[:, None, :, None], k, 0.0)
    q = q.reshape(b, t, hk, hq // hk, d).permute(0, 2, 3, 1, 4).reshape(b, hk, -1, d)
    s = torch.matmul(q, k.transpose(-1, -2)).reshape(b, hk, hq // hk, t, -1) * d ** -0.5
    s = s.masked_fill_(~seen[:, :, None], -math.inf)
    m = s.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, 0.0, m)
    lse = (m + torch.log(torch.exp(s - m).sum(-1, keepdim=True))).squeeze(-1)  # log 0 = -inf for a row that sees nothing
    return s, lse.permute(0, 3, 1, 2).reshape(b, t, hq).contiguous()


def _attend(state):
    s, lse = _scores(state)
    b, hk, grp, t, n = s.shape
    v = torch.where(_visible(state)[1][:, None, :, None], _rows(state["v"], state["table"]), 0.0)
    at = lse.reshape(b, t, hk, grp).permute(0, 2, 3, 1)[..., None]
    p = torch.exp(s - torch.where(at == -math.inf, 0.0, at)).reshape(b, hk, grp * t, n)
    o = torch.matmul(p, v).reshape(b, hk, grp, t, -1).permute(0, 3, 1, 2, 4)
    return {"out": o.reshape(b, t, hk * grp, -1).to(state["q"].dtype), "lse": lse}


def _mass(state):
    s, _ = _scores(state)
    b, hk, grp, t, n = s.shape
    lse = state["lse"].reshape(b, t, hk, grp).permute(0, 2, 3, 1)[..., None]
    p = torch.exp(s - torch.where(lse == -math.inf, 0.0, lse)) * state["weights"][:, None, None, :, None]
    slot = torch.arange(n, device="cuda")[None, None]
    old = torch.where(slot < state["lengths"].long()[:, None, None], state["mass"] * 0.95, 0.0)
    return {"mass": p.sum((2, 3)) + old}


def _append(state):
    q = _rotated(state["q"], state["positions"], state).to(state["q"].dtype)
    k = _rotated(state["knew"], state["positions"], state)
    b, t = state["positions"].shape
    at = torch.arange(t, device="cuda")
    live = at < state["counts"].long()[:, None]
    q = torch.where(live[..., None, None], q, 0.0)
    slot = state["lengths"].long()[:, None] + at
    page = state["k"].shape[2]
    i, j = torch.nonzero(live, as_tuple=True)
    pages, offs = state["table"][i, slot[i, j] // page].long(), slot[i, j] % page
    for pool, new in ((state["k"], k), (state["v"], state["vnew"].float())):
        raw = pool.view(torch.uint8) if pool.dtype == torch.float8_e5m2 else pool
        raw[pages, :, offs] = new[i, j].to(pool.dtype).view(raw.dtype)
    return {"q": q, "k": state["k"], "v": state["v"]}


def _evict(state):
    keep, mass = state["case"]["keep"], state["mass"]
    b, hk, n = mass.shape
    lens = state["lengths"].long()[:, None, None]
    slot = torch.arange(n, device="cuda")[None, None]
    safe = (slot < state["sink"]) | (slot >= lens - state["recent"])
    key = torch.where(slot < lens, torch.where(safe, math.inf, mass), -math.inf)
    order = torch.sort(key, dim=-1, descending=True, stable=True).indices[..., :keep]
    if keep > n:
        order = torch.cat((order, order.new_full((b, hk, keep - n), n)), -1)
    count = lens.clamp_max(keep)
    rank = torch.arange(keep, device="cuda")
    kept = torch.where(rank < count, order, n).sort(-1).values  # ascending slots, the unused ones behind
    live = kept < n
    at = torch.where(live, kept, 0)
    page = state["k"].shape[2]
    pages = state["table"].long()[torch.arange(b, device="cuda")[:, None, None], at // page]
    head = torch.arange(hk, device="cuda")[None, :, None]
    rows = []
    for pool in (state["k"], state["v"]):
        raw = pool.view(torch.uint8) if pool.dtype == torch.float8_e5m2 else pool
        rows.append(torch.where(live[..., None], raw[pages, head, at % page], 0).view(pool.dtype))
    return {"k": rows[0], "v": rows[1], "mass": torch.where(live, mass.gather(-1, at), 0.0),
            "kept": torch.where(live, kept, -1).to(torch.int32), "lengths": count.flatten().to(torch.int32)}


# -------------------------------------------------------------------- a pass

def run(state):
    op = state["case"]["op"]
    if not own:
        if op == "rotary":
            x = state["x"]
            return {"y": _rotated(x, state["positions"], state).to(x.dtype),
                    "grad": _rotated(state["grad"], state["positions"], state, True).to(x.dtype)}
        return {"append": _append, "attend": _attend, "mass": _mass, "evict": _evict}[op](state)
    import lossless_bf16_exponent_gb300 as uz

    if op == "rotary":
        return {"y": uz.rotary(state["x"], state["positions"], state["plan"]),
                "grad": uz.rotary_backward(state["grad"], state["positions"], state["plan"])}
    cache = state["cache"]
    if op == "append":
        q = uz.rotary_append(state["q"], state["knew"], state["vnew"], state["positions"], state["plan"], cache,
                             counts=state["counts"])
        return {"q": q, "k": state["k"], "v": state["v"]}
    if op == "attend":
        out, lse = uz.tree_attention(state["q"], cache, state["mask"], counts=state["counts"])
        return {"out": out, "lse": lse}
    if op == "mass":
        return {"mass": uz.attention_mass(state["q"], cache, state["lse"], state["mask"], counts=state["counts"],
                                          weights=state["weights"], mass=state["mass"], decay=0.95)}
    packed = uz.evict(cache, state["mass"], state["case"]["keep"], sink=state["sink"], recent=state["recent"])
    return {"k": packed.k, "v": packed.v, "mass": packed.mass, "kept": packed.kept, "lengths": packed.lengths}


# ------------------------------------------------------------ the definition

def _turned(x, positions, case, sign):
    """Pair i of each head turned by sign * position * rate_i, in 64 bits."""
    rates, factor = _freqs(case)
    a = positions.double()[..., None, None] * torch.tensor(rates, dtype=torch.float64, device="cuda")
    z = torch.polar(torch.full_like(a, factor), sign * a)
    y, half, rd = x.double().clone(), case["rd"] // 2, case["rd"]
    lo, hi = (slice(0, half), slice(half, rd)) if case["layout"] == "half" else (slice(0, rd, 2), slice(1, rd, 2))
    w = torch.complex(x[..., lo].double(), x[..., hi].double()) * z
    y[..., lo], y[..., hi] = w.real, w.imag
    return y


def exact(case, seed):
    state = prepare(case, seed)
    op = case["op"]
    if op == "rotary":
        return {"y": _turned(state["x"], state["positions"], case, 1.0),
                "grad": _turned(state["grad"], state["positions"], case, -1.0)}
    lens, counts = _lengths(case)
    page = case["page"]

    def tokens(pool, i, upto):
        got = pool[state["table"][i, :-(-upto // page)].long()] if pool.dtype != torch.float8_e5m2 else \
            pool.view(torch.uint8)[state["table"][i, :-(-upto // page)].long()].view(pool.dtype)
        return got.transpose(0, 1).reshape(case["hk"], -1, case["d"])[:, :upto]

    if op == "append":
        q = _turned(state["q"], state["positions"], case, 1.0)
        k, v = _turned(state["knew"], state["positions"], case, 1.0), state["vnew"].double()
        pools = [state["k"].double(), state["v"].double()]
        for i in range(case["b"]):
            q[i, counts[i]:] = 0
            at = torch.arange(lens[i], lens[i] + counts[i], device="cuda")
            where = state["table"][i].long()[at // page]
            pools[0][where, :, at % page] = k[i, :counts[i]]
            pools[1][where, :, at % page] = v[i, :counts[i]]
        return {"q": q, "k": pools[0], "v": pools[1]}
    if op in ("attend", "mass"):
        b, t, hq, d = state["q"].shape
        hk = case["hk"]
        out = torch.zeros((b, t, hq, d), dtype=torch.float64, device="cuda")
        lse = torch.full((b, t, hq), -math.inf, dtype=torch.float64, device="cuda")
        got = torch.zeros((b, hk, _capacity(case)), dtype=torch.float64, device="cuda")
        bits = state["mask"].cpu().numpy().astype(np.uint64)[:, :, 0]
        for i in range(b):
            n, c = lens[i], counts[i]
            if op == "mass":
                got[i, :, :n] = state["mass"][i, :, :n].double() * 0.95
            if not c:
                continue
            sees = torch.ones((c, n + c), dtype=torch.bool)
            for r in range(c):
                for j in range(c):
                    sees[r, n + j] = bool((int(bits[i, r]) >> j) & 1)
            sees = sees.cuda()
            k, v = tokens(state["k"], i, n + c).double(), tokens(state["v"], i, n + c)
            for h in range(hq):
                s = state["q"][i, :c, h].double() @ k[h * hk // hq].T / math.sqrt(d)
                s.masked_fill_(~sees, -math.inf)
                if op == "attend":
                    lse[i, :c, h] = torch.logsumexp(s, -1)
                    out[i, :c, h] = torch.softmax(s, -1) @ v[h * hk // hq].double()
                else:
                    p = torch.exp(s - state["lse"][i, :c, h, None].double())
                    got[i, h * hk // hq, :n + c] += state["weights"][i, :c].double() @ p
        return {"out": out, "lse": lse} if op == "attend" else {"mass": got}
    keep, hk, d = case["keep"], case["hk"], case["d"]
    rows = [torch.zeros((case["b"], hk, keep, d), dtype=torch.float64, device="cuda") for _ in range(2)]
    kept = np.full((case["b"], hk, keep), -1, dtype=np.int32)
    mass = np.zeros((case["b"], hk, keep))
    given = state["mass"].double().cpu().numpy()
    for i, n in enumerate(lens):
        if not n:
            continue
        k, v = tokens(state["k"], i, n).double(), tokens(state["v"], i, n).double()
        for h in range(hk):
            key = given[i, h, :n].copy()
            key[:state["sink"]] = math.inf
            key[max(0, n - state["recent"]):] = math.inf
            at = np.sort(np.lexsort((np.arange(n), -key))[:keep])
            kept[i, h, :at.size], mass[i, h, :at.size] = at, given[i, h, at]
            to = torch.from_numpy(at).cuda()
            rows[0][i, h, :at.size], rows[1][i, h, :at.size] = k[h, to], v[h, to]
    return {"k": rows[0], "v": rows[1], "mass": mass, "kept": kept,
            "lengths": np.array([min(n, keep) for n in lens], dtype=np.int32)}
