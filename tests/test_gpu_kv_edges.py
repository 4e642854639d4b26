"""The KV-cache operators at the edges of what they take: layouts, sizes and
values that the other tests do not reach."""
import math

import pytest
import torch

import test_gpu_kv as K
from test_gpu_kv import BF, DEV, E5, HF, check_attention, gen, make_cache, randn

pytestmark = pytest.mark.gpu


def test_mass_of_any_strides(uz):
    g = gen(1)
    cache = make_cache(uz, g, [200, 90], 2, 2, 64, 16, BF)
    q = randn(g, 2, 2, 4, 64, dtype=BF)
    _, lse = uz.tree_attention(q, cache)
    old = torch.rand(2, 2, cache.capacity, generator=g, device=DEV)
    want = uz.attention_mass(q, cache, lse, mass=old, decay=0.5)
    padded = torch.full((2, 2, cache.capacity + 9), 7.0, device=DEV)
    padded[:, :, 4:-5] = old
    turned = old.transpose(0, 2).contiguous().transpose(0, 2)
    for m in (padded[:, :, 4:-5], turned):
        assert torch.equal(uz.attention_mass(q, cache, lse, mass=m, decay=0.5), want)
        assert torch.equal(m, old)
        box = torch.zeros(2, 3, cache.capacity, device=DEV)
        assert torch.equal(uz.attention_mass(q, cache, lse, mass=m, decay=0.5, out=box[:, 1:]), want)
        assert torch.all(box[:, 0] == 0)


def test_tree_mask_does_not_wait_for_the_stream(uz):
    parents = [[-1, 0, 0, 1, -1, 4]] * 3
    want = uz.tree_mask(parents, device="cpu")
    assert torch.equal(uz.tree_mask(parents).cpu(), want)
    x = torch.zeros(1 << 28, device=DEV)
    done = torch.cuda.Event()
    torch.cuda.synchronize()
    for _ in range(400):  # of a GB each: some 100 ms of work
        x.add_(1.0)
    done.record()
    mask = uz.tree_mask(parents)
    assert not done.query(), "the call waited for the work before it"
    assert torch.equal(mask.cpu(), want) and mask.device == x.device


def test_tree_mask_refuses_a_capture(uz):
    side = torch.cuda.Stream()
    x = torch.zeros(4, device=DEV)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        x.add_(1.0)
        with pytest.raises(ValueError, match="capture"):
            uz.tree_mask([[-1, 0]])
    graph.replay()
    torch.cuda.synchronize()
    assert torch.all(x == 1)


# -------------------------------------------------- bfloat16 queries over an FP8 cache

@pytest.mark.parametrize("t", [1, 3, 24, 70])  # few rows, more, and the tensor-core kernel
@pytest.mark.parametrize("gain,key,scale", [(2.0 ** 126, 2.0 ** -12, 2.0 ** -116), (2.0 ** -130, 2.0 ** 10, 2.0 ** 119)])
def test_queries_at_the_ends_of_bfloat16_over_an_fp8_cache(uz, t, gain, key, scale):
    """The largest and the subnormal bfloat16 numbers lie outside binary16's range, in which the products are taken: a
    power of two out of each row brings them in."""
    g = gen(t)
    cache = make_cache(uz, g, [100, 9], t, 1, 64, 16, E5, scale=key)
    x = randn(g, 2, t, 3, 64)
    q = (x.clamp(-1.9, 1.9) * gain).to(BF)
    q[0, 0, 0, 5] = float(torch.tensor(1.9, dtype=BF)) * gain  # a row whose largest element is 2^126 or above
    q[1, 0, 1] = 0.0  # a row of zeros
    assert torch.isfinite(q).all() and float(q.abs().max()) > gain
    if gain > 1:
        q[0, t - 1, 1, 7] = 3.0e38  # ... and 2^127 or above
    _, lse = check_attention(uz, q, cache, None, [t, t], None, scale=scale)
    mass = uz.attention_mass(q, cache, lse, scale=scale)
    assert float(mass.double().sum()) == pytest.approx(2 * t * 3, rel=1e-3)


def test_queries_with_an_infinity_over_an_fp8_cache(uz):
    cache = make_cache(uz, gen(2), [50], 2, 1, 64, 16, E5)
    q = randn(gen(3), 1, 2, 3, 64, dtype=BF)
    want, _ = uz.tree_attention(q, cache)
    q[0, 1, 2, 9] = math.inf
    out, lse = uz.tree_attention(q, cache)
    assert torch.equal(out[0, 0], want[0, 0]) and torch.equal(out[0, 1, :2], want[0, 1, :2])
    assert not torch.isfinite(lse[0, 1, 2])


# ------------------------------------------------------------ strides of nothing

def test_strides_of_dimensions_of_one_do_not_count(uz):
    """A dimension of one element may have any stride: it is never taken."""
    g = gen(4)

    def odd(x):  # the same elements; dimensions of one get a stride that no alignment allows
        return x.as_strided(x.shape, [3 if n == 1 else s for n, s in zip(x.shape, x.stride())])

    k, v = randn(g, 1, 1, 64, 128, dtype=BF), randn(g, 1, 1, 64, 128, dtype=BF)
    table, lengths = torch.zeros(1, 1, dtype=torch.int32, device=DEV), torch.tensor([40], dtype=torch.int32, device=DEV)
    plain = uz.KVCache(k.clone(), v.clone(), table, lengths)
    cache = uz.KVCache(odd(k), odd(v), table, lengths)
    plan, pos = uz.rotary_plan(128), torch.full((1, 1), 40, dtype=torch.int32, device=DEV)
    for heads in (1, 4):
        q, new = randn(g, 1, 1, heads, 128, dtype=BF), randn(g, 1, 1, 1, 128, dtype=BF)
        want = uz.rotary_append(q, new, new, pos, plan, plain)
        got = uz.rotary_append(odd(q), odd(new), odd(new), pos, plan, cache, out=odd(torch.empty_like(q)))
        assert torch.equal(got, want) and torch.equal(cache.k, plain.k) and torch.equal(cache.v, plain.v)
        assert torch.equal(uz.rotary(odd(q), pos, plan), want)
        out, lse = uz.tree_attention(want, plain)
        got, got_lse = uz.tree_attention(odd(want), cache, out=odd(torch.empty_like(q)))
        assert torch.equal(got, out) and torch.equal(got_lse, lse)
        mass = uz.attention_mass(want, plain, lse)
        assert torch.equal(uz.attention_mass(odd(want), cache, lse, mass=odd(torch.zeros_like(mass))), mass)
    many = randn(g, 1, 40, 4, 128, dtype=BF)  # many rows: pages by tensor maps
    lengths.fill_(20)
    assert torch.equal(uz.tree_attention(odd(many), cache)[0], uz.tree_attention(many, plain)[0])
    assert torch.equal(uz.evict(cache, mass, 1).k, uz.evict(plain, mass, 1).k)
    one = odd(torch.empty(1, 1, 1, 128, dtype=BF, device=DEV))
    assert torch.equal(uz.evict(cache, mass, 1, out_k=one, out_v=odd(torch.empty_like(one))).k, uz.evict(plain, mass, 1).k)


# --------------------------------------- variants that the other sizes do not reach

WIDE = [  # heads above 128: lengths, t, hq, hk, d, page; up to 16 rows, up to 32, more; mass in one chunk and in several
    ([300, 5, 0], 1, 8, 2, 256, 16), ([77, 400], 3, 10, 2, 192, 48), ([129], 2, 2, 1, 144, 400), ([64, 63, 1], 1, 16, 1, 160, 7),
    ([90, 257], 9, 8, 4, 256, 7), ([500], 4, 16, 2, 176, 64), ([33], 32, 2, 2, 144, 16), ([1000, 31], 5, 12, 2, 256, 64),
    ([260, 3], 40, 16, 4, 256, 64), ([129], 150, 2, 1, 192, 16), ([70], 256, 2, 1, 144, 32)]


@pytest.mark.parametrize("q_type,c_type", K.TYPES)
@pytest.mark.parametrize("lens,t,hq,hk,d,page", WIDE)
def test_wide_heads(uz, lens, t, hq, hk, d, page, q_type, c_type):
    K.test_attention(uz, lens, t, hq, hk, d, page, q_type, c_type)
    K.test_mass(uz, lens, t, hq, hk, d, page, q_type, c_type)


@pytest.mark.parametrize("q_type,c_type", [(BF, BF), (HF, HF)])
@pytest.mark.parametrize("lens,t,hq,hk,d,page", [([300, 17], 1, 4, 2, 136, 16), ([200], 6, 8, 2, 248, 64), ([65], 70, 2, 1, 200, 24)])
def test_wide_heads_off_sixteen(uz, lens, t, hq, hk, d, page, q_type, c_type):
    test_wide_heads(uz, lens, t, hq, hk, d, page, q_type, c_type)


@pytest.mark.parametrize("kind", ["many ties", "spread", "equal", "odd values"])
def test_evict_of_rows_longer_than_shared_memory(uz, kind):
    """So many rows that each has one CTA, of more slots than it holds keys for: masses are read again each pass."""
    lens = [30000, 23553, 29999, 100, 0, 24001, 26000] + [23600 + 31 * i for i in range(13)]
    assert len(lens) * 4 * 2 > torch.cuda.get_device_properties(0).multi_processor_count
    K.test_evict(uz, lens, 2000, 4, 100, 4, 16, 4096, kind, BF)


# ------------------------------------------------------------ eviction and the codec

@pytest.mark.parametrize("c_type", [BF, HF, E5])
def test_packed_caches_go_through_the_codec(uz, c_type):
    """Each type's own encoder: e5m2_encode for E5M2, encode for the 16-bit ones; every bit comes back."""
    g = gen(6)
    cache = make_cache(uz, g, [700, 500], 0, 2, 64, 16, c_type)
    mass = torch.rand(2, 2, cache.capacity, generator=g, device=DEV)
    both = torch.empty(2, 2, 2, 128, 64, dtype=c_type, device=DEV)
    uz.evict(cache, mass, 128, sink=4, recent=32, out_k=both[0], out_v=both[1])
    want = both.view(torch.uint8).flatten()
    if c_type == E5:
        stream, n = uz.e5m2_encode(both, uz.e5m2_calibrate(both))
        got = uz.e5m2_decode(stream, both.numel(), stream_bytes=n)
    else:
        stream, n = uz.encode(both, uz.calibrate(both))
        got = uz.decode(stream, both.numel(), stream_bytes=n, dtype=c_type).view(torch.uint8)
    assert torch.equal(got.flatten(), want)
    if c_type != HF:  # FP16's five exponent bits are not where the codebook of bfloat16's eight looks
        assert n < want.numel()


# ------------------------------------------------------------------ outputs in place

@pytest.mark.parametrize("lens,t,hq", [([20, 300], 1, 8), ([9000], 1, 8), ([700, 33], 4, 8), ([40], 30, 8), ([5000, 3], 30, 16), ([100], 200, 16)])
def test_attention_in_place(uz, lens, t, hq):
    """out may be q: rows are read before they are written, whoever else works on their unit."""
    cache = make_cache(uz, gen(t), lens, t, 2, 64, 16, BF)
    box = randn(gen(1), len(lens), t, hq + 2, 64, dtype=BF)
    q = box[:, :, :hq]
    want, lse = uz.tree_attention(q, cache)
    rest = box[:, :, hq:].clone()
    out, got = uz.tree_attention(q, cache, out=q)
    assert out is q and torch.equal(q, want) and torch.equal(got, lse) and torch.equal(box[:, :, hq:], rest)
