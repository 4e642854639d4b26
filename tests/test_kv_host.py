"""Checks of the KV-cache operators that need no GPU: the library exports what
include/uzip_kv.h declares, refuses bad arguments on the host before any CUDA
call (the addresses below are never dereferenced), and the helpers that make
tree masks and rotary rates give what their definitions say."""
import ctypes
import math
import os
import re

import pytest
import torch

import lossless_bf16_exponent_gb300 as uz
from lossless_bf16_exponent_gb300 import _lib, build, kv

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def lib():
    build.build()
    return _lib.load()


def test_exports_match_the_header(lib):
    text = open(os.path.join(ROOT, "include", "uzip_kv.h")).read()
    declared = set(re.findall(r"UZIP_API\s+[\w\s\*]+?\b(uzkv_\w+)\s*\(", text))
    assert declared == set(_lib.KV_EXPORTS)
    nm = os.popen(f"nm -D --defined-only {_lib.lib_path()}").read()
    exported = {line.split()[-1] for line in nm.splitlines() if " T " in line}
    assert {s for s in exported if s.startswith("uzkv_")} == declared


def test_structures_have_the_c_sizes(lib, tmp_path):
    import shutil
    import subprocess

    cc = shutil.which("gcc") or shutil.which("cc")
    if cc is None:
        pytest.skip("no C compiler")
    src = tmp_path / "s.c"
    src.write_text('#include "uzip_kv.h"\n#include <stdio.h>\n'
                   'int main(void) { printf("%zu %zu", sizeof(uzkv_cache_t), sizeof(uzkv_rows_t)); return 0; }\n')
    exe = str(tmp_path / "s")
    subprocess.run([cc, "-std=c11", "-Wall", "-Werror", "-I", os.path.join(ROOT, "include"), str(src), "-o", exe], check=True)
    got = subprocess.run([exe], capture_output=True, text=True).stdout.split()
    assert [int(v) for v in got] == [ctypes.sizeof(_lib.KvCache), ctypes.sizeof(_lib.KvRows)]


A, MIS = 0x10000, 0x10008


def cache(**kw):
    d = dict(d_k=A, d_v=A, k_page_stride=8192, k_head_stride=1024, k_token_stride=64, v_page_stride=8192,
             v_head_stride=1024, v_token_stride=64, d_table=A, table_stride=4, d_lengths=A, d_status=None, pages=10,
             kv_heads=2, page_tokens=16, head_dim=64, sequences=3, pages_per_sequence=4, dtype=0, reserved=0)
    d.update(kw)
    return ctypes.byref(_lib.KvCache(**d))


def rows(d=A, b=4096, t=512, h=64):
    return ctypes.byref(_lib.KvRows(d, b, t, h))


BAD_CACHES = [(dict(d_k=None), "ARG"), (dict(d_v=None), "ARG"), (dict(d_table=None), "ARG"), (dict(d_lengths=None), "ARG"),
              (dict(dtype=2), "ARG"), (dict(dtype=9), "ARG"), (dict(head_dim=60), "ARG"), (dict(head_dim=0), "ARG"),
              (dict(head_dim=264), "ARG"), (dict(pages=0), "ARG"), (dict(page_tokens=0), "ARG"),
              (dict(page_tokens=1 << 20, pages_per_sequence=1 << 12), "ARG"), (dict(k_page_stride=-8), "ARG"),
              (dict(k_token_stride=60), "ALIGN"), (dict(v_head_stride=1023), "ALIGN"), (dict(d_k=MIS), "ALIGN"),
              (dict(d_v=MIS), "ALIGN"), (dict(d_table=A + 2), "ALIGN"), (dict(d_lengths=A + 1), "ALIGN"),
              (dict(d_status=A + 2), "ALIGN"), (dict(sequences=65536), "ARG"), (dict(table_stride=-1), "ARG")]


@pytest.mark.parametrize("kw,want", BAD_CACHES)
def test_every_call_refuses_a_bad_cache(lib, kw, want):
    code = getattr(_lib, "ERR_" + want)
    c = cache(**kw)
    dtype = 0
    assert lib.uzkv_rotary_append(rows(), rows(), rows(), rows(), dtype, 4, 4, A, 4, A, 64, 0, 1.0, None, c, None) == code
    assert lib.uzkv_tree_attention(rows(), rows(), A, dtype, 4, 4, None, 0, None, 1.0, c, A, 1 << 40, None) == code
    assert lib.uzkv_attention_mass(rows(), A, dtype, 4, 4, None, 0, None, None, 1.0, c, None, 1.0, A, 128, 64, 64, None) == code
    assert lib.uzkv_evict(c, A, 128, 64, 64, 8, 1, 1, rows(), rows(), A, A, A, None) == code


def test_rotary_refusals(lib):
    def call(x=rows(), y=rows(), dtype=0, b=2, t=3, h=4, d=64, pos=A, ps=3, turns=A, rd=64, layout=0):
        return lib.uzkv_rotary(x, y, dtype, b, t, h, d, pos, ps, turns, rd, layout, 1.0, 0, None)

    for kw in (dict(x=None), dict(x=rows(None)), dict(y=rows(None)), dict(x=rows(b=-1)), dict(dtype=3), dict(b=0), dict(t=0),
               dict(h=0), dict(d=0), dict(d=257), dict(pos=None), dict(ps=-1), dict(turns=None), dict(rd=0), dict(rd=63),
               dict(rd=66), dict(layout=2)):
        assert call(**kw) == _lib.ERR_ARG, kw
    for kw in (dict(x=rows(A + 1)), dict(y=rows(A + 1)), dict(pos=A + 2), dict(turns=A + 4)):
        assert call(**kw) == _lib.ERR_ALIGN, kw


def test_attention_and_mass_refusals(lib):
    def attend(q=rows(), out=rows(), lse=A, dtype=0, t=4, h=4, mask=None, ms=0, counts=None, c=cache(), ws=A, wb=1 << 40):
        return lib.uzkv_tree_attention(q, out, lse, dtype, t, h, mask, ms, counts, 1.0, c, ws, wb, None)

    def mass(q=rows(), lse=A, dtype=0, t=4, h=4, mask=None, ms=0, counts=None, weights=None, c=cache(), old=None, out=A,
             sb=128, sh=64, slots=64):
        return lib.uzkv_attention_mass(q, lse, dtype, t, h, mask, ms, counts, weights, 1.0, c, old, 1.0, out, sb, sh, slots, None)

    for f in (attend, mass):
        for kw in (dict(q=None), dict(q=rows(None)), dict(dtype=1), dict(dtype=2), dict(dtype=3), dict(t=0), dict(t=257),
                   dict(h=0), dict(h=5), dict(ms=-1), dict(c=None)):
            assert f(**kw) == _lib.ERR_ARG, kw
        for kw in (dict(q=rows(MIS)), dict(q=rows(h=60)), dict(mask=A + 4), dict(counts=A + 2), dict(lse=A + 2)):
            assert f(**kw) == _lib.ERR_ALIGN, kw
    assert attend(out=None) == attend(ws=None) == _lib.ERR_ARG
    assert attend(out=rows(MIS)) == attend(ws=MIS) == _lib.ERR_ALIGN
    need = lib.uzkv_tree_attention_workspace_bytes(3, 4, 4, 2, 64)
    assert need > 0 and attend(wb=need - 1) == _lib.ERR_CAPACITY
    assert lib.uzkv_tree_attention_workspace_bytes(3, 0, 4, 2, 64) == 0
    assert lib.uzkv_tree_attention_workspace_bytes(3, 4, 5, 2, 64) == 0
    for kw in (dict(lse=None), dict(out=None), dict(sb=-1), dict(slots=0), dict(slots=65)):
        assert mass(**kw) == _lib.ERR_ARG, kw
    for kw in (dict(out=A + 2), dict(old=A + 1), dict(weights=A + 2)):
        assert mass(**kw) == _lib.ERR_ALIGN, kw


def test_evict_refusals(lib):
    def call(c=cache(), m=A, sb=128, sh=64, slots=64, keep=8, sink=1, recent=1, k=rows(), v=rows(), kept=A, mo=A, lo=A):
        return lib.uzkv_evict(c, m, sb, sh, slots, keep, sink, recent, k, v, kept, mo, lo, None)

    for kw in (dict(c=None), dict(m=None), dict(sb=-1), dict(slots=0), dict(keep=0), dict(sink=8), dict(recent=9),
               dict(sink=0xFFFFFFFF, recent=2), dict(k=None), dict(v=rows(None)), dict(kept=None), dict(mo=None), dict(lo=None),
               dict(keep=1 << 28)):
        assert call(**kw) == _lib.ERR_ARG, kw
    for kw in (dict(k=rows(MIS)), dict(v=rows(h=60)), dict(m=A + 2), dict(kept=A + 1), dict(lo=A + 2)):
        assert call(**kw) == _lib.ERR_ALIGN, kw


def test_tree_mask_is_the_ancestors():
    parents = [[-1, 0, 0, 1, -1, 4], [-1, -1, -1, 0, 3, 4]]
    m = uz.tree_mask(parents, device="cpu")
    assert m.shape == (2, 6, 1) and m.dtype == torch.int64
    assert m[0, :, 0].tolist() == [0b1, 0b11, 0b101, 0b1011, 0b10000, 0b110000]
    assert m[1, :, 0].tolist() == [0b1, 0b10, 0b100, 0b1001, 0b11001, 0b111001]


def test_tree_mask_passes_a_word():
    m = uz.tree_mask([list(range(-1, 129))], device="cpu")  # a chain of 130
    assert m.shape == (1, 130, 3)
    for t in (0, 62, 63, 64, 127, 128, 129):
        bits = sum((int(w) & ((1 << 64) - 1)) << 64 * i for i, w in enumerate(m[0, t].tolist()))
        assert bits == (1 << (t + 1)) - 1


@pytest.mark.parametrize("bad", [[], [[]], [[0]], [[-1, 2]], [[-2]], [[-1], [-1, 0]], [[-1] * 257]])
def test_tree_mask_refuses(bad):
    with pytest.raises(ValueError):
        uz.tree_mask(bad, device="cpu")


def test_rotary_rates():
    f, m = uz.rotary_rates(8, 10000.0)
    assert m == 1.0 and f == pytest.approx([1.0, 0.1, 0.01, 0.001], rel=1e-14)
    assert uz.rotary_rates(8, scaling="linear", factor=4.0)[0] == pytest.approx([0.25, 0.025, 0.0025, 0.00025], rel=1e-14)
    f, _ = uz.rotary_rates(8, scaling="base", factor=4.0)
    assert f[0] == 1.0 and f[3] == pytest.approx(0.001 / 4.0, rel=1e-12)  # the slowest pair is stretched by the factor
    f, m = uz.rotary_rates(8, scaling="ramp", factor=4.0, original_length=1000, low=1.0, high=32.0)
    assert m == pytest.approx(0.1 * math.log(4.0) + 1)
    turns = [1000 * r / (2 * math.pi) for r in (1.0, 0.1, 0.01, 0.001)]  # 159, 15.9, 1.59, 0.159
    g = [(t - 1) / 31 for t in turns]
    assert f == pytest.approx([1.0, 0.1 * (g[1] + (1 - g[1]) / 4), 0.01 * (g[2] + (1 - g[2]) / 4), 0.00025], rel=1e-12)
    for kw in (dict(rotary_dim=3), dict(rotary_dim=0), dict(rotary_dim=258), dict(rotary_dim=8, scaling="other"),
               dict(rotary_dim=8, factor=0.5), dict(rotary_dim=8, base=1.0), dict(rotary_dim=8, scaling="ramp"),
               dict(rotary_dim=2, scaling="base")):
        with pytest.raises(ValueError):
            uz.rotary_rates(**kw)
    with pytest.raises(ValueError):
        uz.rotary_plan(8, layout="other", device="cpu")
    p = uz.rotary_plan(8, device="cpu")
    assert p.turns.tolist() == [round(r / (2 * math.pi) * 2.0 ** 64) for r in (1.0, 0.1, 0.01, 0.001)]


def test_front_end_refuses_host_tensors():
    x = torch.zeros(2, 3, 4, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        uz.rotary(x, torch.zeros(2, 3, dtype=torch.int32), uz.rotary_plan(64, device="cpu"))
    with pytest.raises(ValueError):
        uz.KVCache(x, x, torch.zeros(2, 1, dtype=torch.int32), torch.zeros(2, dtype=torch.int32))


def test_outputs_may_not_overlap():
    x = torch.zeros(64)
    kv._writable(x.view(4, 16), "out")
    kv._writable(x.view(4, 16)[:, :8].transpose(0, 1), "out")
    for bad in (x[:16].expand(4, 16), x.as_strided((4, 16), (8, 1))):
        with pytest.raises(ValueError):
            kv._writable(bad, "out")
