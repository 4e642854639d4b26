"""The KV-cache operators on the GPU against their definitions in 64 bits, at
the sizes and masks where they can go wrong.

Bounds. u is the unit roundoff of a type (2^-9 bfloat16, 2^-12 ... halves of the
spacing at 1): every result is rounded once to its type, which allows u |y| (2 u
taken). Rotary: the phase is exact to 2^-32 of a turn and rounded to 24 bits of
half a turn, sine and cosine are good to 2 units in the last place: below 2^-20,
2^-19 taken, of |a| + |b|. Scores: products of 16-bit values are exact in 32
bits, a sum of d of them is off by at most d 2^-24 sum |q k| and tensor cores
may cut instead of round: 4 d 2^-24 sum |q k| scale taken, e below. A weight is
then off by the factor exp(2 e) plus 2^-20 for the exponential, and is rounded
to the 16 bits of the values' product (2 u again, of p |v|); an attention output
is a weighted mean of values, so it is off by that factor of sum p |v|.
Weights below the smallest 16-bit number are lost: 2^-24 of |v| each, against
the largest weight."""
import math
import random

import pytest
import torch

pytestmark = pytest.mark.gpu

UNIT = {torch.bfloat16: 2.0 ** -9, torch.float16: 2.0 ** -12, torch.float32: 2.0 ** -25}
BF, HF, F32, E5 = torch.bfloat16, torch.float16, torch.float32, torch.float8_e5m2
DEV = "cuda"


def gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def randn(g, *shape, dtype=F32):
    return torch.randn(shape, generator=g, device=DEV).to(dtype)


# ----------------------------------------------------------------- rotary

def rotary_want(x, pos, rates, factor, rd, layout, sign=1.0):
    a = pos.double()[..., None, None] * torch.tensor(rates, dtype=torch.float64, device=DEV)
    c, s = factor * a.cos(), sign * factor * a.sin()
    x = x.double()
    lo, hi = (slice(0, rd // 2), slice(rd // 2, rd)) if layout == "half" else (slice(0, rd, 2), slice(1, rd, 2))
    y, bound = x.clone(), torch.zeros_like(x)
    y[..., lo] = x[..., lo] * c - x[..., hi] * s
    y[..., hi] = x[..., hi] * c + x[..., lo] * s
    bound[..., lo] = bound[..., hi] = factor * 2.0 ** -19 * (x[..., lo].abs() + x[..., hi].abs())
    return y, bound


SCALINGS = [dict(), dict(scaling="linear", factor=4.0), dict(scaling="base", factor=8.0),
            dict(scaling="ramp", factor=16.0, original_length=4096)]
ROTARY = [  # tokens, heads, d, rd
    (1, 1, 2, 2), (1, 1, 64, 64), (3, 5, 128, 128), (17, 72, 128, 64), (33, 3, 80, 80), (5, 7, 80, 40), (9, 2, 96, 48),
    (7, 3, 256, 256), (4, 3, 257 - 1, 32), (6, 2, 66, 30), (2, 3, 7, 6), (1000, 1, 64, 16), (11, 130, 64, 64), (257, 9, 72, 72)]


@pytest.mark.parametrize("dtype", [BF, HF, F32])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("n,heads,d,rd", ROTARY)
def test_rotary_and_its_gradient(uz, n, heads, d, rd, layout, dtype):
    kw = SCALINGS[(n + heads + d) % 4] if rd > 2 else {}
    rates, factor = uz.rotary_rates(rd, **kw)
    plan = uz.rotary_plan(rd, layout=layout, **kw)
    g = gen(n * d + heads)
    x = randn(g, n, heads, d, dtype=dtype)
    pos = torch.randint(0, 1 << 17, (n,), generator=g, device=DEV).to(torch.int32)
    for f, sign in ((uz.rotary, 1.0), (uz.rotary_backward, -1.0)):
        want, bound = rotary_want(x, pos, rates, factor, rd, layout, sign)
        got = f(x, pos, plan)
        assert got.dtype == dtype and got.shape == x.shape
        assert torch.all((got.double() - want).abs() <= bound + 2 * UNIT[dtype] * want.abs() + 2.0 ** -25)
        assert torch.equal(got[..., rd:], x[..., rd:])


@pytest.mark.parametrize("offset", [0, 1, 4])
def test_rotary_of_views_and_in_place(uz, offset):
    # heads of a fused projection; an offset that leaves rows off every vector boundary
    plan = uz.rotary_plan(64, layout="half")
    rates, factor = uz.rotary_rates(64)
    base = randn(gen(5), 3 * 9 * 7 * 64 + 8, dtype=BF)
    x = base[offset:offset + 3 * 9 * 7 * 64].view(3, 9, 7, 64)[:, :, 2:6]
    pos = torch.arange(27, device=DEV, dtype=torch.int32).view(3, 9) * 1000
    want, bound = rotary_want(x, pos, rates, factor, 64, "half")
    before = base.clone()
    got = uz.rotary(x, pos, plan)
    assert torch.all((got.double() - want).abs() <= bound + 2 * UNIT[BF] * want.abs())
    assert torch.equal(base, before)
    assert uz.rotary(x, pos, plan, out=x) is x
    assert torch.equal(x, got)
    rest = torch.ones_like(base, dtype=torch.bool)
    rest[offset:offset + 3 * 9 * 7 * 64].view(3, 9, 7, 64)[:, :, 2:6] = False
    assert torch.equal(base[rest], before[rest])


def test_rotary_far_positions(uz):
    rates, factor = uz.rotary_rates(128)
    pos = torch.tensor([0, 1, 131071, 1 << 20, (1 << 31) - 1], device=DEV, dtype=torch.int32)
    x = randn(gen(6), 5, 2, 128)
    want, bound = rotary_want(x, pos, rates, factor, 128, "half")
    got = uz.rotary(x, pos, uz.rotary_plan(128))
    # 2^31 positions times a rate known to 2^-54 of itself: 2^-20 radians more on either side
    assert torch.all((got.double() - want).abs() <= 4 * bound + 2 * UNIT[F32] * want.abs())
    assert torch.equal(got[0], x[0])


def test_rotary_gradient_against_differences(uz):
    plan = uz.rotary_plan(48, layout="interleaved", scaling="ramp", factor=8.0, original_length=512)
    g = gen(7)
    x, w = randn(g, 13, 3, 96), randn(g, 13, 3, 96)
    pos = torch.randint(0, 5000, (13,), generator=g, device=DEV).to(torch.int32)
    grad = uz.rotary_backward(w, pos, plan).double()
    f = lambda z: (uz.rotary(z, pos, plan).double() * w.double()).sum()
    for k in range(8):
        u = randn(g, 13, 3, 96)
        diff = (f(x + u) - f(x - u)) / 2  # the map is linear: the step need not be small
        size = w.double().norm() * (x.double().norm() + u.double().norm()) * plan.magnitude
        assert abs(diff - (grad * u.double()).sum()) <= 2.0 ** -18 * size


def test_rotary_of_nothing_and_special_values(uz):
    plan = uz.rotary_plan(4)
    assert uz.rotary(torch.empty(0, 3, 8, device=DEV), torch.empty(0, dtype=torch.int32, device=DEV), plan).shape == (0, 3, 8)
    x = torch.ones(2, 1, 8, device=DEV)
    x[0, 0, 6] = math.nan
    x[0, 0, 7] = math.inf  # in the part that is not turned: copied
    y = uz.rotary(x, torch.tensor([3, 4], dtype=torch.int32, device=DEV), plan)
    assert torch.isnan(y[0, 0, 6]) and y[0, 0, 7] == math.inf and torch.isfinite(y[0, 0, :6]).all() and torch.isfinite(y[1]).all()


# ------------------------------------------------------------------ caches

def make_cache(uz, g, lens, extra, hk, d, page, dtype, form="pool", status=None, scale=1.0):
    """A cache of random pages; slots that no sequence uses are NaN. extra: room for new tokens."""
    b = len(lens)
    per = max(1, -(-(max(lens) + extra) // page))
    pages = b * per + 2
    table = (torch.randperm(pages, generator=g, device=DEV)[:b * per]).view(b, per).to(torch.int32)
    full = lambda *s: torch.full(s, math.nan, device=DEV).to(dtype)
    if form == "pool":  # K and V pages side by side
        pool = full(pages, 2, hk, page, d)
        k, v = pool[:, 0], pool[:, 1]
    elif form == "tokens":  # heads within a token, rows longer than the head
        k, v = (full(pages, page, hk, d + 16)[..., :d].transpose(1, 2) for _ in range(2))
    else:
        raise ValueError(form)
    n = max(lens) + extra
    for i in range(b):
        for j0 in range(0, lens[i] + extra, page):
            m = min(page, lens[i] + extra - j0)
            p = int(table[i, j0 // page])
            k[p, :, :m] = (randn(g, hk, m, d) * scale).to(dtype)
            v[p, :, :m] = randn(g, hk, m, d).to(dtype)
        table[i, -(-(lens[i] + extra) // page):] = -1  # never read
    lengths = torch.tensor(lens, dtype=torch.int32, device=DEV)
    return uz.KVCache(k, v, table, lengths, status=status)


def raw(x):
    return x.view(torch.uint8) if x.dtype == E5 else x


def cached(cache, i, upto, which="k"):
    """[heads, upto, dim] of sequence i, float64."""
    pool = getattr(cache, which)
    page = pool.shape[2]
    m = -(-upto // page)
    if not m:
        return torch.empty(pool.shape[1], 0, pool.shape[3], dtype=torch.float64, device=DEV)
    got = torch.cat([pool[int(p)].double() for p in cache.page_table[i, :m]], 1)
    return got[:, :upto]


# ------------------------------------------------------------------ append

APPEND = [  # b, t, hq, hk, d, rd, page, counts
    (1, 1, 1, 1, 64, 64, 16, None), (3, 5, 8, 2, 128, 128, 16, [5, 0, 3]), (2, 33, 5, 5, 80, 40, 7, None),
    (4, 2, 24, 8, 96, 96, 1, [2, 1, 2, 0]), (2, 70, 6, 3, 256, 64, 48, [70, 69])]


@pytest.mark.parametrize("form", ["pool", "tokens"])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("dtype,ctype", [(BF, BF), (HF, HF), (BF, E5), (HF, E5)])
@pytest.mark.parametrize("b,t,hq,hk,d,rd,page,counts", APPEND)
def test_append(uz, b, t, hq, hk, d, rd, page, counts, dtype, ctype, layout, form):
    g = gen(b * t + d)
    lens = [17 * i % 40 for i in range(b)]
    cache = make_cache(uz, g, lens, t, hk, d, page, ctype, form)
    k0, v0 = raw(cache.k).clone(), raw(cache.v).clone()
    qkv = randn(g, b, t, hq + 2 * hk, d, dtype=dtype)
    pos = torch.randint(0, 1 << 17, (b, t), generator=g, device=DEV).to(torch.int32)
    rates, factor = uz.rotary_rates(rd)
    c = torch.tensor(counts, dtype=torch.int32, device=DEV) if counts else None
    q = uz.rotary_append(qkv[:, :, :hq], qkv[:, :, hq:hq + hk], qkv[:, :, hq + hk:], pos,
                         uz.rotary_plan(rd, layout=layout), cache, counts=c)
    live = counts or [t] * b
    want, bound = rotary_want(qkv[:, :, :hq + hk], pos, rates, factor, rd, layout)
    e5 = 2.0 ** -3 if ctype == E5 else 2 * UNIT[dtype]
    written = torch.zeros(k0.shape[0], page, dtype=torch.bool, device=DEV)
    for i in range(b):
        m = live[i]
        w, e = want[i, :m, :hq], bound[i, :m, :hq]
        assert torch.all((q[i, :m].double() - w).abs() <= e + 2 * UNIT[dtype] * w.abs() + 2.0 ** -25)
        assert torch.all(q[i, m:] == 0)
        for u in range(m):
            p, o = int(cache.page_table[i, (lens[i] + u) // page]), (lens[i] + u) % page
            written[p, o] = True
            w, e = want[i, u, hq:], bound[i, u, hq:]
            assert torch.all((cache.k[p, :, o].double() - w).abs() <= e + e5 * w.abs() + 2.0 ** -17)
            assert torch.equal(raw(cache.v[p, :, o].contiguous()), raw(qkv[i, u, hq + hk:].to(ctype).contiguous()))
    same = ~written[:, None, :, None].expand(k0.shape)
    nan = torch.iinfo(torch.uint8) if ctype == E5 else None
    bits = lambda x: x if nan else x.contiguous().view(torch.int16)
    assert torch.equal(bits(raw(cache.k))[same], bits(k0)[same]) and torch.equal(bits(raw(cache.v))[same], bits(v0)[same])


def test_append_rounds_to_e5m2_as_the_type(uz):
    # every binary16 pattern as a value: stored as torch rounds it, overflow to infinity, NaN to NaN
    x = torch.arange(65536, device=DEV, dtype=torch.int32).to(torch.int16).view(HF).view(1, 512, 1, 128)
    k, v = (torch.zeros(1, 1, 512, 128, device=DEV).to(E5) for _ in range(2))
    cache = uz.KVCache(k, v, torch.zeros(1, 1, dtype=torch.int32, device=DEV), torch.zeros(1, dtype=torch.int32, device=DEV))
    uz.rotary_append(x, x, x, torch.zeros(1, 512, dtype=torch.int32, device=DEV), uz.rotary_plan(2), cache)
    want = x.view(512, 128).float().to(E5).float()
    got = v.view(512, 128).float()
    assert torch.equal(torch.isnan(got), torch.isnan(want))
    fine = ~torch.isnan(want)
    assert torch.equal(got[fine], want[fine])


# --------------------------------------------------------------- attention

def mask_bits(mask, i, c, t):
    """bool [c, c] of sequence i."""
    if mask is None:
        return torch.tril(torch.ones(c, c, dtype=torch.bool, device=DEV))
    row = mask[i if mask.shape[0] > 1 else 0].cpu().tolist()
    return torch.tensor([[bool((row[r][u // 64] >> (u % 64)) & 1) for u in range(c)] for r in range(c)],
                        dtype=torch.bool, device=DEV).view(c, c)


def attention_want(q, cache, mask, live, scale):
    """(out, bound, lse, bound, per-row data) in float64."""
    b, t, hq, d = q.shape
    grp = hq // cache.kv_heads
    lens = cache.lengths.tolist()
    u16 = UNIT[HF] if cache.dtype == E5 else UNIT[q.dtype]
    out = torch.zeros(b, t, hq, d, dtype=torch.float64, device=DEV)
    ob, lse = torch.zeros_like(out), torch.full((b, t, hq), -math.inf, dtype=torch.float64, device=DEV)
    lb = torch.zeros_like(lse)
    for i in range(b):
        n, c = lens[i], live[i]
        if not c:
            continue
        k, v = cached(cache, i, n + c), cached(cache, i, n + c, "v")
        sees = torch.cat((torch.ones(c, n, dtype=torch.bool, device=DEV), mask_bits(mask, i, c, t)), 1)
        for h in range(hq):
            qq, kk, vv = q[i, :c, h].double(), k[h // grp], v[h // grp]
            s = (qq @ kk.T * scale).masked_fill(~sees, -math.inf)
            size = (qq.abs() @ kk.abs().T * abs(scale)).masked_fill(~sees, 0).amax(-1)
            e = 4 * d * 2.0 ** -24 * size
            some = sees.any(-1)
            l = torch.logsumexp(s, -1)
            p = torch.where(sees, torch.exp(s - torch.where(some, l, 0.0)[:, None]), 0.0)
            top = p.amax(-1, keepdim=True)
            # a value that a row does not see has no part in it, whatever it is
            o = torch.stack([(p[r, sees[r]][:, None] * vv[sees[r]]).sum(0) for r in range(c)])
            mean = torch.stack([(p[r, sees[r]][:, None] * vv[sees[r]].abs()).sum(0) for r in range(c)])
            lost = torch.stack([vv[sees[r]].abs().sum(0) for r in range(c)]) * top * 2.0 ** -24
            out[i, :c, h] = torch.where(some[:, None], o, 0.0)
            lse[i, :c, h] = l
            ob[i, :c, h] = ((torch.expm1(4 * e) + 2.0 ** -18)[:, None] + 2 * u16) * mean + lost + 2 * UNIT[q.dtype] * o.abs() + 2.0 ** -24
            lb[i, :c, h] = 2 * e + 2.0 ** -20 * (1 + torch.where(some, l, 0.0).abs())
    return out, ob, lse, lb


def check_attention(uz, q, cache, mask, live, counts, scale=None, **kw):
    d = q.shape[3]
    out, lse = uz.tree_attention(q, cache, mask, counts=counts, scale=scale, **kw)
    want, ob, wl, lb = attention_want(q, cache, mask, live, d ** -0.5 if scale is None else scale)
    fin = torch.isfinite(want)
    assert torch.equal(torch.isfinite(out), fin)
    bad = (out.double() - want).abs()[fin] > ob[fin]
    assert not bad.any(), f"{int(bad.sum())} of {bad.numel()} outputs, worst {float(((out.double() - want).abs()[fin] / ob[fin]).max())} of the bound"
    empty = wl == -math.inf
    assert torch.equal(lse == -math.inf, empty)
    f = torch.isfinite(wl)
    assert torch.all((lse.double() - wl).abs()[f] <= lb[f])
    assert torch.all(out[empty] == 0)
    return out, lse


def random_tree(uz, seed, b, t):
    r = random.Random(seed)
    return uz.tree_mask([[r.randint(max(-1, i - 4), i - 1) if i else -1 for i in range(t)] for _ in range(b)])


TYPES = [(BF, BF), (HF, HF), (BF, E5), (HF, E5)]
SHAPES = [  # lengths, t, hq, hk, d, page
    ([0], 1, 1, 1, 64, 16), ([1], 1, 8, 8, 128, 16), ([15, 16, 17], 1, 4, 2, 64, 16), ([63, 64, 65, 0], 2, 8, 1, 128, 64),
    ([127, 129], 3, 10, 2, 80, 48), ([200, 31], 5, 14, 2, 96, 7), ([1000, 5], 1, 64, 8, 128, 16), ([333], 16, 16, 2, 128, 1),
    ([130, 77, 9], 17, 5, 1, 64, 400), ([512], 33, 6, 3, 256, 32), ([70, 300], 64, 8, 4, 128, 16), ([90], 65, 4, 2, 64, 16),
    ([257], 130, 16, 2, 128, 64), ([11], 256, 3, 1, 128, 16), ([4097], 1, 16, 1, 128, 64), ([3000, 100, 0, 1, 2, 2999], 4, 8, 2, 64, 16),
    ([20, 3], 7, 34, 2, 16, 5), ([600], 2, 26, 2, 48, 33)]


@pytest.mark.parametrize("q_type,c_type", TYPES)
@pytest.mark.parametrize("lens,t,hq,hk,d,page", SHAPES)
def test_attention(uz, lens, t, hq, hk, d, page, q_type, c_type):
    g = gen(sum(lens) + t * d)
    b = len(lens)
    cache = make_cache(uz, g, lens, t, hk, d, page, c_type, ["pool", "tokens"][(t + d // 16) % 2])
    q = randn(g, b, t, hq, d, dtype=q_type)
    live = [t - (i * 3) % (t + 1) for i in range(b)]
    counts = torch.tensor(live, dtype=torch.int32, device=DEV)
    check_attention(uz, q, cache, random_tree(uz, t, b, t), live, counts)
    check_attention(uz, q, cache, None, [t] * b, None)


@pytest.mark.parametrize("q_type,c_type", TYPES)
def test_attention_peaked_and_flat_scores(uz, q_type, c_type):
    g = gen(3)
    for scale in (0.0, 1e-3, 1.0, -0.5, 4.0):  # scores to about 200: one key holds the row
        cache = make_cache(uz, g, [700, 50], 3, 2, 128, 16, c_type, scale=1.5)
        q = randn(g, 2, 3, 8, 128, dtype=q_type)
        check_attention(uz, q, cache, None, [3, 3], None, scale=scale)


def test_attention_rising_and_falling_maxima(uz):
    # the largest score moves from tile to tile, up or down: the running maximum is rescaled every time or never
    for sign in (1.0, -1.0):
        cache = make_cache(uz, gen(4), [1500], 1, 1, 64, 32, BF)
        ramp = torch.linspace(0, 30, 1501, device=DEV) * sign
        for j in range(1501):
            cache.k[int(cache.page_table[0, j // 32]), 0, j % 32] = ramp[j].to(BF)
        q = torch.full((1, 1, 4, 64), 1 / 8, device=DEV, dtype=BF)
        check_attention(uz, q, cache, None, [1], None)


@pytest.mark.parametrize("q_type,c_type", TYPES)
@pytest.mark.parametrize("t", [1, 3, 16, 64, 100])
def test_attention_rows_that_see_nothing(uz, t, q_type, c_type):
    cache = make_cache(uz, gen(8), [0, 40], t, 2, 64, 16, c_type)
    q = randn(gen(9), 2, t, 4, 64, dtype=q_type)
    mask = torch.zeros(1, t, -(-t // 64), dtype=torch.int64, device=DEV)
    mask[0, t // 2, 0] = 1  # one row sees the first new token
    check_attention(uz, q, cache, mask, [t, t], None)


@pytest.mark.parametrize("q_type,c_type", TYPES)
@pytest.mark.parametrize("what", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("t,n", [(4, 0), (4, 13), (20, 100), (70, 60)])
def test_attention_keeps_out_what_is_masked(uz, t, n, what, q_type, c_type):
    """A new token whose key and value are not finite touches only the rows that see it."""
    g = gen(t + n)
    hq, hk, d = 6, 2, 64
    clean = make_cache(uz, g, [n], t, hk, d, 16, c_type)
    q = randn(g, 1, t, hq, d, dtype=q_type)
    parents = [[-1] * t]  # every node is a root: it sees the cache and itself
    mask = uz.tree_mask(parents)
    want, wl = uz.tree_attention(q, clean, mask)
    for part in "kv":
        dirty = make_cache(uz, gen(t + n), [n], t, hk, d, 16, c_type)
        bad = [1, t - 1]
        for u in bad:
            getattr(dirty, part)[int(dirty.page_table[0, (n + u) // 16]), :, (n + u) % 16] = what
        got, gl = uz.tree_attention(q, dirty, mask)
        fine = [u for u in range(t) if u not in bad]
        assert torch.equal(got[:, fine], want[:, fine]) and torch.equal(gl[:, fine], wl[:, fine])
        if part == "v":
            assert torch.equal(gl, wl) and not torch.isfinite(got[:, bad]).any()
            if not math.isnan(what) and n == 0:
                assert torch.all(got[:, bad] == what)
    nan_q = q.clone()
    nan_q[0, 2] = math.nan
    got, gl = uz.tree_attention(nan_q, clean, mask)
    fine = [u for u in range(t) if u != 2]
    assert torch.equal(got[:, fine], want[:, fine]) and torch.isnan(got[:, 2]).all() and torch.isnan(gl[:, 2]).all()


def test_attention_of_nan_in_the_cache(uz):
    cache = make_cache(uz, gen(1), [300], 2, 2, 64, 16, BF)
    cache.v[int(cache.page_table[0, 5]), 1, 3, 7] = math.nan  # one element of one head's value
    q = randn(gen(2), 1, 2, 4, 64, dtype=BF)
    out, lse = uz.tree_attention(q, cache)
    bad = torch.isnan(out)
    assert bad[0, :, 2:, 7].all() and int(bad.sum()) == 4 and torch.isfinite(lse).all()


@pytest.mark.parametrize("t", [1, 24])
def test_attention_of_large_queries_over_an_fp8_cache(uz, t):
    # bfloat16 queries beyond and below binary16's range: scores stay right
    for gain in (2.0 ** 40, 2.0 ** -40):
        cache = make_cache(uz, gen(11), [100], t, 1, 64, 16, E5)
        q = (randn(gen(12), 1, t, 3, 64) * gain).to(BF)
        check_attention(uz, q, cache, None, [t], None, scale=0.1 / gain)


def test_attention_strides_streams_and_given_buffers(uz):
    g = gen(13)
    cache = make_cache(uz, g, [500, 333], 5, 2, 128, 16, BF)
    qkv = randn(g, 2, 5, 12, 128, dtype=BF)
    q = qkv[:, :, 2:10]
    want, wl = check_attention(uz, q, cache, None, [5, 5], None)
    box = torch.full((2, 5, 10, 128), 7.0, device=DEV, dtype=BF)
    lse = torch.empty(2, 5, 8, device=DEV)
    ws = torch.full((uz.tree_attention_workspace_bytes(cache, 5, 8),), 0xFF, dtype=torch.uint8, device=DEV)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        out, l2 = uz.tree_attention(q, cache, out=box[:, :, 1:9], lse=lse, workspace=ws)
    side.synchronize()
    assert torch.equal(out, want) and torch.equal(l2, wl) and l2 is lse
    assert torch.all(box[:, :, 0] == 7) and torch.all(box[:, :, 9] == 7)
    # transposed queries [heads, tokens], and a query that is one row repeated
    qt = q.transpose(1, 2).contiguous().transpose(1, 2)
    assert torch.equal(uz.tree_attention(qt, cache)[0], want)
    one = q[:, :, :1].expand(-1, -1, 8, -1)
    same = uz.tree_attention(one, cache)[0]
    assert torch.equal(same, uz.tree_attention(one.contiguous(), cache)[0])


def test_attention_repeats_bit_for_bit(uz):
    cache = make_cache(uz, gen(14), [9000, 12, 4000], 9, 4, 64, 16, BF)
    q = randn(gen(15), 3, 9, 16, 64, dtype=BF)
    first = uz.tree_attention(q, cache)
    for _ in range(5):
        again = uz.tree_attention(q, cache)
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])


def test_contiguous_cache_is_pages_of_whole_sequences(uz):
    g = gen(16)
    k, v = randn(g, 3, 2, 100, 64, dtype=HF), randn(g, 3, 2, 100, 64, dtype=HF)
    table = torch.arange(3, dtype=torch.int32, device=DEV)[:, None]
    cache = uz.KVCache(k, v, table, torch.tensor([97, 10, 99], dtype=torch.int32, device=DEV))
    check_attention(uz, randn(g, 3, 1, 4, 64, dtype=HF), cache, None, [1, 1, 1], None)


def test_pool_beyond_32_bit_offsets(uz):
    pages, page, d = 9000, 4096, 128  # 4.7 G elements a pool
    pool = torch.empty(pages, 1, page, d, dtype=BF, device=DEV)
    table = torch.tensor([[pages - 1, 17], [8200, pages - 2]], dtype=torch.int32, device=DEV)
    g = gen(17)
    for p in table.flatten().tolist():
        pool[p] = randn(g, 1, page, d, dtype=BF)
    cache = uz.KVCache(pool, pool, table, torch.tensor([5000, 4100], dtype=torch.int32, device=DEV))
    q = randn(g, 2, 1, 2, d, dtype=BF)
    _, lse = check_attention(uz, q, cache, None, [1, 1], None)
    m = uz.attention_mass(q, cache, lse)
    assert torch.all((m.double().sum(-1) - 2).abs() < 1e-3)
    packed = uz.evict(cache, m, 64)
    for i in range(2):
        rows = cached(cache, i, 5000 if i == 0 else 4100)[0]
        assert torch.equal(packed.k[i, 0].double(), rows[packed.kept[i, 0].long()])
    pos = torch.zeros(2, 1, dtype=torch.int32, device=DEV)  # keys and values share the pool: both write the same row
    new = randn(g, 2, 1, 1, d, dtype=BF)
    uz.rotary_append(q, new, new, pos, uz.rotary_plan(2), cache)
    assert torch.equal(pool[17, 0, 5000 - 4096], new[0, 0, 0]) and torch.equal(pool[pages - 2, 0, 4], new[1, 0, 0])


# -------------------------------------------------------------------- mass

@pytest.mark.parametrize("q_type,c_type", TYPES)
@pytest.mark.parametrize("lens,t,hq,hk,d,page", SHAPES)
def test_mass(uz, lens, t, hq, hk, d, page, q_type, c_type):
    g = gen(sum(lens) + t * d + 1)
    b = len(lens)
    cache = make_cache(uz, g, lens, t, hk, d, page, c_type, ["pool", "tokens"][(t + d // 16) % 2])
    q = randn(g, b, t, hq, d, dtype=q_type)
    live = [t - (i * 3) % (t + 1) for i in range(b)]
    counts = torch.tensor(live, dtype=torch.int32, device=DEV)
    mask = random_tree(uz, t, b, t)
    lse = attention_want(q, cache, mask, live, d ** -0.5)[2].float()
    weights = (torch.rand(b, t, generator=g, device=DEV) < 0.7).float() * 0.5
    old = torch.rand(b, hk, cache.capacity, generator=g, device=DEV)
    for w, m, c, mk in ((weights, old, counts, mask), (None, None, None, None)):
        lv = live if c is not None else [t] * b
        if mk is None:
            lse = attention_want(q, cache, None, lv, d ** -0.5)[2].float()
        got = uz.attention_mass(q, cache, lse, mk, counts=c, weights=w, mass=m, decay=0.75)
        for i in range(b):
            n, cc = lens[i], lv[i]
            k = cached(cache, i, n + cc)
            want = torch.zeros(hk, n + cc, dtype=torch.float64, device=DEV)
            bound = torch.zeros_like(want)
            if m is not None:
                want[:, :n] = 0.75 * m[i, :, :n].double()
            if cc:
                sees = torch.cat((torch.ones(cc, n, dtype=torch.bool, device=DEV), mask_bits(mk, i, cc, t)), 1)
                for h in range(hq):
                    kk, qq = k[h // (hq // hk)], q[i, :cc, h].double()
                    s = qq @ kk.T * d ** -0.5
                    e = 4 * d * 2.0 ** -24 * (qq.abs() @ kk.abs().T) * d ** -0.5
                    at = lse[i, :cc, h, None].double()
                    p = torch.where(sees & (at != -math.inf), torch.exp(s - torch.where(at == -math.inf, 0.0, at)), 0.0)
                    p = p * (w[i, :cc, None].double() if w is not None else 1.0)
                    want[h // (hq // hk)] += p.sum(0)
                    # the exponent's argument and log weight are rounded to 24 bits of at most |s| + |lse|
                    bound[h // (hq // hk)] += (p * (torch.expm1(2 * e) + 2.0 ** -22 * (s.abs() + at.abs().clamp_max(1e3)) + 2.0 ** -18)).sum(0)
            far = (got[i, :, :n + cc].double() - want).abs()
            assert torch.all(far <= bound + 2.0 ** -21 * want + 1e-30), float((far / (bound + 1e-30)).max())
            assert torch.all(got[i, :, n + cc:] == 0)


def test_mass_in_place_narrow_and_strided(uz):
    g = gen(18)
    cache = make_cache(uz, g, [200, 90], 2, 2, 64, 16, BF)
    q = randn(g, 2, 2, 4, 64, dtype=BF)
    _, lse = uz.tree_attention(q, cache)
    want = uz.attention_mass(q, cache, lse)
    box = torch.rand(2, 2, 300, generator=g, device=DEV)
    keep = box.clone()
    part = box[:, :, 7:7 + 150]
    assert uz.attention_mass(q, cache, lse, mass=part, decay=0.5, out=part) is part
    old = torch.where(torch.arange(150, device=DEV) < cache.lengths[:, None, None], keep[:, :, 7:157] * 0.5, 0.0)
    assert torch.allclose(part, want[:, :, :150] + old, rtol=2.0 ** -20, atol=0)
    assert torch.equal(box[:, :, :7], keep[:, :, :7]) and torch.equal(box[:, :, 157:], keep[:, :, 157:])


def test_mass_ignores_rows_that_saw_nothing_and_masked_nans(uz):
    t = 6
    cache = make_cache(uz, gen(19), [0, 30], t, 1, 64, 16, BF)
    q = randn(gen(20), 2, t, 2, 64, dtype=BF)
    mask = torch.zeros(1, t, 1, dtype=torch.int64, device=DEV)
    mask[0, 3, 0] = 1 << 3
    cache.k[int(cache.page_table[1, 31 // 16]), :, 31 % 16] = math.nan  # new token 1, seen by none
    _, lse = uz.tree_attention(q, cache, mask)
    m = uz.attention_mass(q, cache, lse, mask)
    assert torch.isfinite(m).all()
    assert float(m[0, 0, 3]) == pytest.approx(2.0, rel=1e-4) and float(m[0].sum()) == pytest.approx(2.0, rel=1e-4)
    assert float(m[1].sum()) == pytest.approx(12.0, rel=1e-3)


# ------------------------------------------------------------------- evict

def evict_want(mass, n, keep, sink, recent):
    """Kept slots of one row, by sorting (class, mass, slot)."""
    vals = mass[:n].double().cpu().tolist()
    rank = [(0 if (j < sink or j >= n - recent) else 2 if math.isnan(x) else 1, 0.0 if math.isnan(x) or j < sink or j >= n - recent else -x, j)
            for j, x in enumerate(vals)]
    return sorted(j for _, _, j in sorted(rank)[:keep])


EVICT = [  # lengths, keep, sink, recent, hk, d, page
    ([1], 1, 0, 0, 1, 64, 16), ([0, 5, 4], 4, 0, 0, 2, 64, 16), ([100, 99, 3], 10, 2, 3, 2, 128, 16), ([1000, 17], 100, 0, 100, 1, 80, 7),
    ([5000, 2500, 0], 1111, 4, 200, 3, 64, 48), ([70000], 3000, 4, 1000, 2, 64, 64), ([40000, 39999], 39999, 0, 0, 1, 64, 400),
    ([257] * 5, 256, 1, 0, 8, 96, 1), ([9000], 1, 1, 0, 1, 256, 16), ([64], 200, 3, 5, 2, 64, 16)]


@pytest.mark.parametrize("c_type", [BF, E5])
@pytest.mark.parametrize("kind", ["many ties", "spread", "equal", "odd values"])
@pytest.mark.parametrize("lens,keep,sink,recent,hk,d,page", EVICT)
def test_evict(uz, lens, keep, sink, recent, hk, d, page, kind, c_type):
    g = gen(sum(lens) + keep)
    b = len(lens)
    cache = make_cache(uz, g, lens, 0, hk, d, page, c_type)
    u = torch.rand(b, hk, cache.capacity, generator=g, device=DEV)
    if kind == "many ties":
        mass = (u * 4).floor() / 4
    elif kind == "spread":
        mass = torch.exp(40 * u - 20)
    elif kind == "equal":
        mass = torch.full_like(u, 0.125)
    else:
        odd = torch.tensor([math.nan, -math.nan, math.inf, -math.inf, 0.0, -0.0, -1.5, 1e-45, -1e-45, 3e38], device=DEV)
        mass = odd[(u * 10).long().clamp_max(9)]
    for i in range(b):
        mass[i, :, lens[i]:] = math.nan  # never read
    got = uz.evict(cache, mass, keep, sink=sink, recent=recent)
    assert got.lengths.tolist() == [min(n, keep) for n in lens]
    for i in range(b):
        m = min(lens[i], keep)
        k, v = cached(cache, i, lens[i]), cached(cache, i, lens[i], "v")
        for h in range(hk):
            want = evict_want(mass[i, h], lens[i], keep, sink, recent)
            assert got.kept[i, h].tolist() == want + [-1] * (keep - m)
            at = torch.tensor(want, dtype=torch.long, device=DEV)
            assert torch.equal(got.k[i, h, :m].double(), k[h, at]) and torch.equal(got.v[i, h, :m].double(), v[h, at])
            assert torch.equal(got.mass[i, h, :m].view(torch.int32), mass[i, h, at].view(torch.int32))
            assert torch.all(raw(got.k[i, h, m:]) == 0) and torch.all(raw(got.v[i, h, m:]) == 0) and torch.all(got.mass[i, h, m:] == 0)


def test_evict_into_views_with_room(uz):
    g = gen(21)
    cache = make_cache(uz, g, [300, 250], 0, 2, 64, 16, BF)
    mass = torch.rand(2, 2, cache.capacity + 5, generator=g, device=DEV)[:, :, 3:]
    want = uz.evict(cache, mass, 40, recent=8)
    box = torch.full((2, 2, 2, 64, 64), 7.0, device=DEV, dtype=BF)
    got = uz.evict(cache, mass, 40, recent=8, out_k=box[0][:, :, :40], out_v=box[1][:, :, :40])
    assert torch.equal(got.k, want.k) and torch.equal(got.v, want.v) and torch.all(box[:, :, :, 40:] == 7)


# ------------------------------------------------- what only the device sees

def test_lengths_and_pages_out_of_range_are_reported(uz):
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    g = gen(22)
    cache = make_cache(uz, g, [30, 20], 2, 2, 64, 16, BF, status=status)
    q = randn(g, 2, 2, 4, 64, dtype=BF)
    pos = torch.zeros(2, 2, dtype=torch.int32, device=DEV)
    new = randn(g, 2, 2, 2, 64, dtype=BF)
    plan = uz.rotary_plan(64)

    def everything():
        uz.rotary_append(q, new, new, pos, plan, cache)
        _, lse = uz.tree_attention(q, cache)
        m = uz.attention_mass(q, cache, lse)
        uz.evict(cache, m, 8)

    calls = [lambda: uz.rotary_append(q, new, new, pos, plan, cache), lambda: uz.tree_attention(q, cache),
             lambda: uz.attention_mass(q, cache, torch.zeros(2, 2, 4, device=DEV)),
             lambda: uz.evict(cache, torch.zeros(2, 2, cache.capacity, device=DEV), 8)]
    everything()
    assert int(status) == 0
    good_lengths, good_table = cache.lengths.clone(), cache.page_table.clone()
    for spoil in (lambda: cache.lengths.fill_(-1), lambda: cache.lengths.fill_(1 << 30), lambda: cache.page_table.fill_(-7),
                  lambda: cache.page_table.fill_(1 << 30)):
        for call in calls:
            status.zero_()
            spoil()
            call()
            assert int(status) == 5
            cache.lengths.copy_(good_lengths)
            cache.page_table.copy_(good_table)
    status.zero_()
    everything()
    assert int(status) == 0


# ---------------------------------------------------------------- refusals

def test_front_end_refusals(uz):
    g = gen(23)
    cache = make_cache(uz, g, [30, 20], 2, 2, 64, 16, BF)
    k, v, table, lengths = cache.k, cache.v, cache.page_table, cache.lengths
    for args in ((k.float(), v.float(), table, lengths), (k, v.to(HF), table, lengths), (k, v[:, :1], table, lengths), (k[0], v[0], table, lengths),
                 (k, v, table.long(), lengths), (k, v, table[0], lengths), (k, v, table, lengths.long()), (k, v, table, lengths[:1]),
                 (k, v, table.cpu(), lengths), (k, v, table.t().contiguous().t(), lengths), (k.transpose(2, 3), v.transpose(2, 3), table, lengths),
                 (k[:1].expand(3, -1, -1, -1), v[:3], table, lengths), (k, v, table, lengths, torch.zeros(2, dtype=torch.int32, device=DEV))):
        with pytest.raises(ValueError):
            uz.KVCache(*args)
    q = randn(g, 2, 2, 4, 64, dtype=BF)
    lse = torch.zeros(2, 2, 4, device=DEV)
    new = q[:, :, :2]
    pos = torch.zeros(2, 2, dtype=torch.int32, device=DEV)
    plan = uz.rotary_plan(64)
    mask = uz.tree_mask([[-1, 0]] * 2)
    one = torch.ones(2, dtype=torch.int32, device=DEV)
    bad_q = [q[:1], q.to(HF), q.float(), q[..., :32], q.cpu(), q[0]]
    for x in bad_q:
        with pytest.raises(ValueError):
            uz.tree_attention(x, cache)
        with pytest.raises(ValueError):
            uz.attention_mass(x, cache, lse)
        with pytest.raises(ValueError):
            uz.rotary_append(x, new, new, pos, plan, cache)
    for kw in (dict(mask=mask[:, :1]), dict(mask=mask.int()), dict(mask=mask[:, :, 0]), dict(mask=mask.expand(2, 2, 1)[:, [0, 1]].cpu()),
               dict(counts=one.long()), dict(counts=one[:1]), dict(out=q[:, :1]), dict(out=q.to(HF)), dict(out=q[:, :, :1].expand(-1, -1, 4, -1)),
               dict(lse=lse[:1]), dict(lse=lse.double()), dict(workspace=torch.zeros(64, device=DEV))):
        with pytest.raises(ValueError):
            uz.tree_attention(q, cache, **kw)
    with pytest.raises(ValueError):
        uz.tree_attention(q[:, :, :3], cache)
    with pytest.raises(ValueError):
        uz.tree_attention(q[:, :0], cache)
    with pytest.raises(uz.UzipError):
        uz.tree_attention(q, cache, workspace=torch.empty(0, dtype=torch.uint8, device=DEV))
    with pytest.raises(uz.UzipError) as e:
        uz.tree_attention(torch.zeros(2 * 2 * 4 * 64 + 8, device=DEV, dtype=BF)[1:1 + 1024].view(2, 2, 4, 64), cache)
    assert e.value.code == 2
    m = torch.zeros(2, 2, cache.capacity, device=DEV)
    for kw in (dict(weights=torch.zeros(2, 3, device=DEV)), dict(mass=m[:, :1]), dict(mass=m.double()), dict(out=m[:1]),
               dict(mass=m, out=torch.zeros(2, 2, 2 * cache.capacity, device=DEV)[..., ::2]), dict(out=torch.zeros(2, 2, cache.capacity + 1, device=DEV))):
        with pytest.raises(ValueError):
            uz.attention_mass(q, cache, lse, **kw)
    for kw in (dict(keep=0), dict(keep=4, sink=3, recent=2), dict(keep=4, sink=-1), dict(keep=4, out_k=torch.zeros(2, 2, 4, 64, device=DEV, dtype=BF)),
               dict(keep=4, mass=m[:1]), dict(keep=4, mass=m.double())):
        with pytest.raises(ValueError):
            uz.evict(cache, **{"mass": m, **kw})
    for args in ((q, pos[:, :1], plan), (q, pos.long(), plan), (q.to(E5), pos, plan), (q[0, 0], pos, plan)):
        with pytest.raises(ValueError):
            uz.rotary(*args)
    with pytest.raises(ValueError):
        uz.rotary(q, pos, plan, out=q[:, :, :1].expand(-1, -1, 4, -1))
    with pytest.raises(uz.UzipError):
        uz.rotary(q, pos, uz.rotary_plan(128))
    for kw in (dict(k=new.to(HF)), dict(v=new[:, :1]), dict(k=q), dict(positions=pos[:1]), dict(counts=one.long()), dict(out=q.to(HF))):
        with pytest.raises(ValueError):
            uz.rotary_append(**{**dict(q=q, k=new, v=new, positions=pos, plan=plan, cache=cache), **kw})
