"""The KV-cache operators together, and the paths their small tests do not
reach: the example's whole round, calls captured in a CUDA graph, many rows over
many tiles with the softmax reference rising at every one, more rows than one
pass takes, both ways of copying pages."""
import importlib.util
import math
import os
import sys

import pytest
import torch

sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))
from test_gpu_kv import BF, E5, HF, attention_want, check_attention, gen, make_cache, randn, random_tree  # noqa: E402

pytestmark = pytest.mark.gpu
DEV = "cuda"
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_example_round(uz):
    spec = importlib.util.spec_from_file_location("serve_drafts", os.path.join(ROOT, "examples", "serve_drafts.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    r = m.main()
    assert r["bit_identical"] and r["finite"]
    assert r["sent_bytes"] < r["kept_bytes"] < r["prompt_bytes"]
    assert m.KEEP / m.PROMPT < r["mass_kept"] < 1.0


@pytest.mark.parametrize("q_type,c_type", [(BF, BF), (HF, HF), (BF, E5)])
@pytest.mark.parametrize("rows", [40, 128, 130, 256, 300])
@pytest.mark.parametrize("page", [16, 64, 24, 7])
def test_many_rows_with_a_rising_reference(uz, page, rows, q_type, c_type):
    """Every tile's scores are far above those before: each is a rescaling, with none or some of the products before
    it still running. The status word stays clear: no wait ran out."""
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    n, d, heads = 1500, 64, 4
    t = -(-rows // heads)
    cache = make_cache(uz, gen(rows + page), [n, 70], t, 1, d, page, c_type, status=status)
    for i in range(2):
        for j in range(0, [n, 70][i] + t):
            p = int(cache.page_table[i, j // page])
            cache.k[p, 0, j % page] = (0.02 * (j // 32)) * torch.ones(d, device=DEV).to(c_type).float()
    q = (0.5 + torch.rand((2, t, heads, d), generator=gen(3), device=DEV)).to(q_type)
    check_attention(uz, q, cache, random_tree(uz, 5, 2, t), [t, t - 1], torch.tensor([t, t - 1], dtype=torch.int32, device=DEV), scale=0.5)
    assert int(status) == 0


@pytest.mark.parametrize("page", [32, 5])
def test_many_sequences_of_many_rows(uz, page):
    """Units of every length side by side: tiles in turn, tiles of both streams, parts and wholes."""
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    lens = [(37 * i) % 700 for i in range(60)]
    cache = make_cache(uz, gen(4), lens, 40, 2, 64, page, BF, status=status)
    for heads in (4, 16):
        q = randn(gen(heads), 60, 40, heads, 64, dtype=BF)
        live = [(i * 7) % 41 for i in range(60)]
        check_attention(uz, q, cache, None, live, torch.tensor(live, dtype=torch.int32, device=DEV))
    assert int(status) == 0


def test_pages_copied_either_way_agree(uz):
    """The same tokens in pages that allow bulk copies and in pages that do not give the same masses and, up to the
    order of parts, the same attention."""
    for c_type, heads in ((BF, 8), (E5, 8), (BF, 64)):
        out = []
        for page in (64, 9):
            g = gen(77)
            cache = make_cache(uz, g, [900], 3, 2, 128, page, c_type)
            rows = randn(gen(78), 2, 903, 128)
            for j in range(903):
                p = int(cache.page_table[0, j // page])
                cache.k[p, :, j % page] = rows[:, j].to(c_type)
                cache.v[p, :, j % page] = (rows[:, j] * 0.5).to(c_type)
            q = randn(gen(79), 1, 3, heads, 128, dtype=BF)
            o, lse = uz.tree_attention(q, cache)
            out.append((o, lse, uz.attention_mass(q, cache, torch.full_like(lse, 3.0), out=torch.empty(1, 2, 903, device=DEV))))
        assert torch.equal(out[0][0], out[1][0]) and torch.equal(out[0][1], out[1][1]) and torch.equal(out[0][2], out[1][2])


def test_calls_in_a_graph(uz):
    g = gen(5)
    cache = make_cache(uz, g, [300, 100], 4, 2, 64, 16, BF)
    qkv = randn(g, 2, 4, 12, 64, dtype=BF)
    pos = torch.arange(8, device=DEV, dtype=torch.int32).view(2, 4)
    plan = uz.rotary_plan(64)

    def step():
        q = uz.rotary_append(qkv[:, :, :8], qkv[:, :, 8:10], qkv[:, :, 10:], pos, plan, cache)
        out, lse = uz.tree_attention(q, cache)
        mass = uz.attention_mass(q, cache, lse)
        return out, mass, uz.evict(cache, mass, 32, recent=4)

    want = step()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert torch.equal(got[2].kept, want[2].kept) and torch.equal(got[2].k, want[2].k)


def test_calls_on_two_streams_and_threads(uz):
    import threading

    cache = make_cache(uz, gen(6), [5000, 3000], 2, 4, 64, 16, BF)
    q = [randn(gen(7 + i), 2, 2, 16, 64, dtype=BF) for i in range(2)]
    want = [uz.tree_attention(x, cache) for x in q]
    torch.cuda.synchronize()
    got: list = [None, None]

    def work(i):
        with torch.cuda.stream(torch.cuda.Stream()):
            for _ in range(50):
                got[i] = uz.tree_attention(q[i], cache)
            torch.cuda.current_stream().synchronize()

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    for i in range(2):
        assert torch.equal(got[i][0], want[i][0]) and torch.equal(got[i][1], want[i][1])


def test_rows_beyond_one_pass(uz):
    # 256 tokens of 16 heads a KV head: 4096 rows, in many row tiles and mass chunks
    cache = make_cache(uz, gen(8), [333], 256, 1, 64, 64, BF)
    q = randn(gen(9), 1, 256, 16, 64, dtype=BF)
    _, lse = check_attention(uz, q, cache, None, [256], None)
    m = uz.attention_mass(q, cache, lse)
    assert float(m.double().sum()) == pytest.approx(4096.0, rel=1e-4)
    want = attention_want(q, cache, None, [256], 64 ** -0.5)[2]
    assert torch.allclose(lse.double(), want, atol=1e-4) and math.isfinite(float(m.max()))
