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
