"""The codec's calls run on their tensors' device, whichever is current (tensors
and library stand in for a GPU's)."""
import pytest
import torch

import lossless_bf16_exponent_gb300 as uz
from lossless_bf16_exponent_gb300 import codec, pipeline
from test_kv_front_end import Bench, OnGpu


class Tensor(OnGpu):
    def reshape(self, *shape):
        return Tensor(self.host.reshape(*shape), self.index)

    def view(self, *a):
        return Tensor(self.host.view(*a), self.index)

    def __getitem__(self, at):
        return Tensor(self.host[at], self.index)


class Recorder(Bench):
    def __init__(self, monkeypatch):
        super().__init__(monkeypatch)
        plain = codec.load()

        class Library:
            def __getattr__(self, name):
                if name.endswith(("compressed_size", "workspace_bytes")):
                    return lambda *args: 64
                return getattr(plain, name)

        library = Library()
        monkeypatch.setattr(codec, "load", lambda: library)
        empty = torch.empty
        monkeypatch.setattr(torch, "empty", lambda *a, **kw: Tensor((t := empty(*a, **kw)).host, t.index))


@pytest.mark.parametrize("index", [0, 1])
def test_codec_calls_run_on_the_tensors_device(monkeypatch, index):
    bench = Recorder(monkeypatch)
    x, bytes8 = Tensor(torch.zeros(256, dtype=torch.bfloat16), index), Tensor(torch.zeros(256, dtype=torch.uint8), index)
    cb, s = Tensor(torch.zeros(4096, dtype=torch.uint8), index), Tensor(torch.zeros(512, dtype=torch.uint8), index)
    side = type("Stream", (), {"device": torch.device("cuda", index), "cuda_stream": 1000 + index})()
    monkeypatch.setattr(torch.cuda, "current_stream", lambda d=None: side)
    calls = [lambda: uz.calibrate(x), lambda: uz.codebook_from_exps(range(16), device=torch.device("cuda", index)), lambda: uz.encode(x, cb),
             lambda: uz.encode_dynamic(x), lambda: uz.decode(s, 16), lambda: uz.stream_copy(s, s), lambda: uz.stream_info(s),
             lambda: uz.e5m2_calibrate(bytes8), lambda: uz.e5m2_encode(bytes8, cb), lambda: uz.e5m2_decode(s, 16),
             lambda: uz.make_sentinel(cb), lambda: uz.sentinel_encode(x, cb), lambda: uz.sentinel_decode(s, 16)]
    for current in (0, 1):
        for call in calls:
            bench.current = current
            bench.calls.clear()
            call()
            assert [d for _, d, _ in bench.calls] == [index] and bench.current == current, bench.calls
            stream = bench.calls[0][2][-1]
            assert getattr(stream, "value", stream) == 1000 + index


def test_the_pipeline_runs_on_the_tensors_device(monkeypatch):
    bench = Recorder(monkeypatch)
    seen = []
    monkeypatch.setattr(pipeline, "split_points", lambda n, pieces: seen.append(bench.current) or 1 / 0)
    monkeypatch.setattr(torch, "empty_like", lambda t: t)
    x = Tensor(torch.zeros(256, dtype=torch.bfloat16), 1)
    with pytest.raises(ZeroDivisionError):
        pipeline.send_compressed(x, None)
    assert seen == [1] and bench.current == 0
