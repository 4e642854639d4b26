"""The front end of the KV-cache operators without a GPU: tensors that stand in
for those of a GPU, and a library that records what reaches it."""
import ctypes

import pytest
import torch

import lossless_bf16_exponent_gb300 as uz
from lossless_bf16_exponent_gb300 import codec, kv


class OnGpu:
    """A host tensor that says it is on a GPU; views of it say the same."""

    def __init__(self, t, index=0):
        self.host, self.index = t, index

    is_cuda = True

    @property
    def device(self):
        return torch.device("cuda", self.index)

    def get_device(self):
        return self.index

    def __getitem__(self, at):
        return OnGpu(self.host[at], self.index)

    def __getattr__(self, name):
        got = getattr(self.host, name)
        if name in ("contiguous", "expand", "view", "copy_", "transpose"):
            def f(*a, **kw):
                got(*(x.host if isinstance(x, OnGpu) else x for x in a), **kw)
                return self if name == "copy_" else OnGpu(got(*a, **kw), self.index)
            return f
        return got


class Bench:
    """A stand-in for the GPUs and the library: `current` is the current device, `calls` what was called with which
    device current."""

    def __init__(self, monkeypatch):
        self.current, self.calls, self.asked = 0, [], []
        bench = self

        class device:
            def __init__(self, d):
                self.to = d if isinstance(d, int) else torch.device(d).index

            def __enter__(self):
                self.back, bench.current = bench.current, self.to

            def __exit__(self, *exc):
                bench.current = self.back

        class Library:
            def __getattr__(self, name):
                def f(*args):
                    if name.endswith("workspace_bytes"):
                        return 64
                    bench.calls.append((name, bench.current, args))
                    return 0
                f.__name__ = name
                return f

        def empty(*shape, dtype=None, device=None, **kw):
            shape = shape[0] if len(shape) == 1 else shape
            return OnGpu(torch.zeros(shape, dtype=dtype), torch.device(device).index)

        def capturing():
            bench.asked.append(bench.current)
            return False

        library = Library()
        monkeypatch.setattr(kv, "load", lambda: library)
        monkeypatch.setattr(codec, "load", lambda: library)
        monkeypatch.setattr(codec, "_raw_stream", lambda i: 1000 + i)
        monkeypatch.setattr(codec, "_current_device", lambda: self.current, raising=False)
        monkeypatch.setattr(torch.cuda, "current_device", lambda: self.current)
        monkeypatch.setattr(torch.cuda, "device", device)
        monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", capturing)
        monkeypatch.setattr(torch, "empty", empty)
        self.bumped = []
        monkeypatch.setattr(kv, "increment_version", self.bumped.extend, raising=False)


@pytest.fixture
def bench(monkeypatch):
    return Bench(monkeypatch)


BF, F32, I32 = torch.bfloat16, torch.float32, torch.int32


def zeros(*shape, dtype=BF, index=0):
    return OnGpu(torch.zeros(shape, dtype=dtype), index)


def make(index=0, b=2, hk=2, page=16, pages=4, d=64):
    pool = zeros(pages, 2, hk, page, d, index=index)
    return uz.KVCache(pool[:, 0], pool[:, 1], zeros(b, 2, dtype=I32, index=index), zeros(b, dtype=I32, index=index))


def plan_on(index, rd=64):
    return uz.RotaryPlan(zeros(rd // 2, dtype=torch.int64, index=index), rd, "half", 1.0)


def every_call(index):
    cache = make(index)
    q, new = zeros(2, 3, 4, 64, index=index), zeros(2, 3, 2, 64, index=index)
    pos, plan = zeros(2, 3, dtype=I32, index=index), plan_on(index)
    lse, mass = zeros(2, 3, 4, dtype=F32, index=index), zeros(2, 2, 32, dtype=F32, index=index)
    return [("uzkv_rotary", lambda: uz.rotary(q, pos, plan)), ("uzkv_rotary", lambda: uz.rotary_backward(q, pos, plan)),
            ("uzkv_rotary_append", lambda: uz.rotary_append(q, new, new, pos, plan, cache)),
            ("uzkv_tree_attention", lambda: uz.tree_attention(q, cache)),
            ("uzkv_attention_mass", lambda: uz.attention_mass(q, cache, lse)), ("uzkv_evict", lambda: uz.evict(cache, mass, 8))]


@pytest.mark.parametrize("index", [0, 1])
def test_calls_run_on_the_tensors_device(bench, index):
    """Each call launches with its tensors' device current and on that device's stream, whatever device is current, and
    leaves the current device as it was."""
    for current in (0, 1):
        for name, call in every_call(index):
            bench.current, bench.calls, bench.asked = current, [], []
            call()
            assert [(n, d) for n, d, _ in bench.calls] == [(name, index)]
            assert bench.calls[0][2][-1] == 1000 + index and bench.current == current
            assert all(d == index for d in bench.asked)


def test_a_cache_keeps_its_tensors(bench):
    """What a call passes on are the addresses taken when the cache was made: its tensors cannot be exchanged under it,
    and advancing them in place goes on to work."""
    cache = make()
    for name in ("k", "v", "page_table", "lengths", "status", "dtype", "capacity", "_c"):
        before = getattr(cache, name)
        with pytest.raises(AttributeError):
            setattr(cache, name, zeros(2, dtype=I32))
        assert getattr(cache, name) is before
    with pytest.raises(AttributeError):
        del cache.lengths
    lengths = torch.zeros(2, dtype=I32)
    cache.lengths.host.copy_(lengths)
    cache.lengths = cache.lengths  # what an in-place operator assigns
    uz.evict(cache, zeros(2, 2, 32, dtype=F32), 8)
    reached = ctypes.cast(bench.calls[0][2][0], ctypes.POINTER(uz._lib.KvCache)).contents
    assert reached.d_lengths == cache.lengths.data_ptr()


def test_a_gradient_is_not_cut_without_a_word(bench):
    """Operators without a gradient refuse inputs whose gradient is being recorded, as does an `out`; without recording
    they take them, and a given output counts as written."""
    cache, pos, plan = make(), zeros(2, 3, dtype=I32), plan_on(0)
    q, new, lse, mass = zeros(2, 3, 4, 64), zeros(2, 3, 2, 64), zeros(2, 3, 4, dtype=F32), zeros(2, 2, 32, dtype=F32)
    weights, out, wide = zeros(2, 3, dtype=F32), zeros(2, 3, 4, 64), zeros(2, 2, 8, 64)
    calls = {
        "q": [lambda: uz.tree_attention(q, cache), lambda: uz.attention_mass(q, cache, lse), lambda: uz.rotary(q, pos, plan, out=out),
              lambda: uz.rotary_append(q, new, new, pos, plan, cache), lambda: uz.rotary_backward(q, pos, plan, out=q)],
        "new": [lambda: uz.rotary_append(q, new, new, pos, plan, cache)],
        "lse": [lambda: uz.attention_mass(q, cache, lse), lambda: uz.tree_attention(q, cache, lse=lse)],
        "weights": [lambda: uz.attention_mass(q, cache, lse, weights=weights)],
        "mass": [lambda: uz.attention_mass(q, cache, lse, mass=mass), lambda: uz.evict(cache, mass, 8)],
        "out": [lambda: uz.rotary(q, pos, plan, out=out), lambda: uz.tree_attention(q, cache, out=out),
                lambda: uz.rotary_append(q, new, new, pos, plan, cache, out=out)],
        "wide": [lambda: uz.evict(cache, mass, 8, out_k=wide, out_v=zeros(2, 2, 8, 64))]}
    named = dict(q=q, new=new, lse=lse, weights=weights, mass=mass, out=out, wide=wide)
    for name, those in calls.items():
        for call in those:
            named[name].host.requires_grad_(True)
            bench.calls.clear()
            with pytest.raises(ValueError, match="gradient"):
                call()
            assert not bench.calls
            with torch.no_grad():
                call()
            named[name].host.requires_grad_(False)
            call()
            assert len(bench.calls) == 2
    pool = zeros(4, 2, 2, 16, 64)
    pool.host.requires_grad_(True)
    with pytest.raises(ValueError):
        uz.KVCache(pool[:, 0], pool[:, 1], zeros(2, 2, dtype=I32), zeros(2, dtype=I32))
    bench.bumped.clear()
    box = zeros(2, 2, 32, dtype=F32)
    uz.rotary(q, pos, plan, out=out)
    uz.rotary(q, pos, plan)
    uz.tree_attention(q, cache, out=out, lse=lse)
    uz.attention_mass(q, cache, lse, out=box)
    assert bench.bumped == [out, out, lse, box]


def test_outputs_may_not_share_memory_with_inputs(bench):
    """An output that overlaps an input without being it is written while it is read: refused. Views side by side in one
    buffer, and an output that is the input, go through."""
    cache, pos, plan = make(), zeros(2, 3, dtype=I32), plan_on(0)
    box = zeros(2, 3, 12, 64)  # heads of a projection
    q, new = box[:, :, :4], box[:, :, 8:10]
    lse, mass = zeros(2, 3, 4, dtype=F32), zeros(2, 2, 40, dtype=F32)
    rows = zeros(2, 2, 24, 64)
    flat = zeros(4 * 6 * 256 + 64)
    shifted, plain = flat[8:8 + 6 * 256].view(2, 3, 4, 64), flat[:6 * 256].view(2, 3, 4, 64)
    bad = [lambda: uz.rotary(q, pos, plan, out=box[:, :, 1:5]), lambda: uz.rotary_backward(plain, pos, plan, out=shifted),
           lambda: uz.rotary_append(q, new, new, pos, plan, cache, out=box[:, :, 3:7]),
           lambda: uz.rotary_append(q, new, box[:, :, 10:12], pos, plan, cache, out=box[:, :, 7:11]),
           lambda: uz.rotary_append(q, new, box[:, :, 10:12], pos, plan, cache, out=box[:, :, 4:12][:, :, 4:8]),
           lambda: uz.tree_attention(q, cache, out=box[:, :, 2:6]),
           lambda: uz.attention_mass(q, cache, lse, mass=mass[:, :, 0:20], out=mass[:, :, 4:24]),
           lambda: uz.attention_mass(q, cache, lse, out=OnGpu(torch.as_strided(lse.host, (2, 2, 4), (8, 4, 1)))),
           lambda: uz.evict(cache, mass, 8, out_k=rows[:, :, :8], out_v=rows[:, :, 7:15]),
           lambda: uz.evict(cache, mass, 8, out_k=cache.k[1:3, :, :8], out_v=rows[:, :, :8]),
           lambda: uz.evict(cache, mass, 8, out_k=rows[:, :, :8], out_v=cache.v[:2, :, 8:])]
    for i, call in enumerate(bad):
        with pytest.raises(ValueError, match="overlap"):
            call()
        assert not bench.calls, i
    good = [lambda: uz.rotary(q, pos, plan, out=q), lambda: uz.rotary(q, pos, plan, out=box[:, :, :4]),
            lambda: uz.rotary(q, pos, plan, out=box[:, :, 4:8]), lambda: uz.rotary(plain, pos, plan, out=flat[6 * 256:12 * 256].view(2, 3, 4, 64)),
            lambda: uz.rotary_append(q, new, box[:, :, 10:12], pos, plan, cache, out=box[:, :, 4:8]),
            lambda: uz.rotary_append(q, new, new, pos, plan, cache, out=q), lambda: uz.tree_attention(q, cache, out=box[:, :, 4:8]),
            lambda: uz.tree_attention(q, cache, out=q), lambda: uz.attention_mass(q, cache, lse, mass=mass[:, :, :20], out=mass[:, :, :20]),
            lambda: uz.attention_mass(q, cache, lse, mass=mass[:, :, :20], out=mass[:, :, 20:]),
            lambda: uz.evict(cache, mass, 8, out_k=rows[:, :, :8], out_v=rows[:, :, 8:16])]
    for call in good:
        call()
    assert len(bench.calls) == len(good)


def test_overlap_of_views_is_exact():
    import random

    r = random.Random(5)
    flat = torch.zeros(400, dtype=torch.int16)
    seen = {True: 0, False: 0}
    for _ in range(4000):
        views = []
        for _ in range(2):
            shape = [r.randint(0 if r.random() < 0.02 else 1, 4) for _ in range(r.randint(1, 4))]
            strides = [r.choice([0, 1, 2, 3, 4, 6, 8, 12, 16, 24, 48]) for _ in shape]
            t = flat if r.random() < 0.8 else flat.view(torch.uint8)
            reach = sum((max(n, 1) - 1) * s for n, s in zip(shape, strides))
            if reach >= 400:
                strides, reach = [1] * len(shape), sum(max(n, 1) - 1 for n in shape)
            views.append(t.as_strided(shape, strides, r.randint(0, min(399 - reach, 60))))
        marks = []
        for v in views:
            base = torch.zeros(800, dtype=torch.uint8)
            offset = v.storage_offset() * v.element_size()
            same = base.as_strided([*v.shape, v.element_size()], [*(s * v.element_size() for s in v.stride()), 1], offset)
            if v.numel():
                same.fill_(1)
            marks.append(base)
        want = bool((marks[0] & marks[1]).any())
        assert kv._overlap(*views) == kv._overlap(*views[::-1]) == want
        seen[want] += 1
    assert min(seen.values()) > 500


def test_mass_of_any_strides(bench):
    """A mass that is a view goes through: strides of dimensions of one element do not count, and one whose rows lie
    otherwise than the output's is copied to the output, which may be both."""
    cache, q, lse = make(b=1), zeros(1, 3, 4, 64), zeros(1, 3, 4, dtype=F32)
    wide = zeros(1, 8, 2, 32, dtype=F32)[:, 0]  # one sequence of a longer buffer
    assert wide.is_contiguous() and wide.stride(0) != 64
    uz.attention_mass(q, cache, lse, mass=wide)
    assert bench.calls[-1][2][11] == wide.data_ptr()
    padded = OnGpu(torch.arange(100, dtype=F32).view(1, 2, 50))[:, :, 3:35]
    out = uz.attention_mass(q, cache, lse, mass=padded)
    args = bench.calls[-1][2]
    assert args[11] == args[13] == out.data_ptr() and args[14:17] == (64, 32, 32)
    assert torch.equal(out.host, padded.host)
    box = zeros(1, 2, 40, dtype=F32)
    turned = OnGpu(torch.arange(64, dtype=F32).view(1, 32, 2).transpose(1, 2))  # rows not contiguous
    assert uz.attention_mass(q, cache, lse, mass=turned, out=box[:, :, 8:]).data_ptr() == box.data_ptr() + 32
    assert torch.equal(box.host[:, :, 8:], turned.host) and torch.all(box.host[:, :, :8] == 0)
    same = zeros(1, 2, 64, dtype=F32)
    uz.attention_mass(q, cache, lse, mass=same[:, :, :32], out=same[:, :, :32])
    assert bench.calls[-1][2][11] == bench.calls[-1][2][13] == same.data_ptr()
    with pytest.raises(ValueError):
        uz.attention_mass(q, cache, lse, mass=same)


def test_append_of_no_heads_is_refused_and_of_no_tokens_is_nothing(bench):
    """Without query heads nothing was stored and nothing said; without tokens there is nothing to store."""
    cache, pos, plan, new = make(), zeros(2, 3, dtype=I32), plan_on(0), zeros(2, 3, 2, 64)
    with pytest.raises(ValueError, match="heads"):
        uz.rotary_append(zeros(2, 3, 0, 64), new, new, pos, plan, cache)
    none = zeros(2, 0, 4, 64)
    assert uz.rotary_append(none, new[:, :0], new[:, :0], pos[:, :0], plan, cache).shape == (2, 0, 4, 64)
    assert not bench.calls


def test_the_ramp_without_its_magnitude():
    """The ramp in turns between 1 and 4 with cosines and sines as they are: a published scaling of long contexts."""
    kw = dict(base=500000.0, scaling="ramp", factor=8.0, original_length=8192, low=1.0, high=4.0)
    rates, factor = uz.rotary_rates(128, **kw, magnitude=1.0)
    assert factor == 1.0 and rates == uz.rotary_rates(128, **kw)[0]
    for i, f in enumerate(rates):
        plain = 500000.0 ** (-2 * i / 128)
        length = 2 * 3.141592653589793 / plain  # positions of a turn
        mix = min(1.0, max(0.0, (8192 / length - 1.0) / 3.0))
        assert f == pytest.approx(plain * (mix + (1 - mix) / 8.0), rel=1e-12)
    assert uz.rotary_plan(128, **kw, magnitude=1.0, device="cpu").magnitude == 1.0
    assert uz.rotary_plan(128, **kw, device="cpu").magnitude == uz.rotary_rates(128, **kw)[1] > 1.2
    assert uz.rotary_rates(8, magnitude=0.5) == (uz.rotary_rates(8)[0], 0.5)
    for bad in (0.0, -1.0, float("nan"), float("inf")):
        with pytest.raises(ValueError):
            uz.rotary_rates(8, magnitude=bad)


def test_a_batch_of_no_sequences_gives_empty_results(bench):
    cache, plan = make(b=0), plan_on(0)
    q, new, pos = zeros(0, 3, 4, 64), zeros(0, 3, 2, 64), zeros(0, 3, dtype=I32)
    assert uz.rotary(q, pos, plan).shape == uz.rotary_append(q, new, new, pos, plan, cache).shape == (0, 3, 4, 64)
    out, lse = uz.tree_attention(q, cache)
    assert out.shape == (0, 3, 4, 64) and lse.shape == (0, 3, 4)
    mass = uz.attention_mass(q, cache, lse)
    assert mass.shape == (0, 2, 32)
    packed = uz.evict(cache, mass, 8)
    assert packed.k.shape == packed.v.shape == (0, 2, 8, 64) and packed.kept.shape == (0, 2, 8) and packed.lengths.shape == (0,)
    assert not bench.calls
