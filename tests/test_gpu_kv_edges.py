"""The KV-cache operators at the edges of what they take: layouts, sizes and
values that the other tests do not reach."""
import math

import pytest
import torch

from test_gpu_kv import BF, DEV, E5, F32, HF, cached, check_attention, evict_want, gen, make_cache, randn, random_tree, raw  # noqa: F401

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
