"""Refusals of the KV-cache operators' C entries that come before any CUDA call
(the addresses below are never dereferenced)."""
import ctypes

import pytest

from lossless_bf16_exponent_gb300 import _lib, build

A = 0x10000


@pytest.fixture(scope="module")
def lib():
    build.build()
    return _lib.load()


def cache(**kw):
    d = dict(d_k=A, d_v=A, k_page_stride=8192, k_head_stride=1024, k_token_stride=64, v_page_stride=8192,
             v_head_stride=1024, v_token_stride=64, d_table=A, table_stride=4, d_lengths=A, d_status=None, pages=10,
             kv_heads=2, page_tokens=16, head_dim=64, sequences=3, pages_per_sequence=4, dtype=0, reserved=0)
    d.update(kw)
    return ctypes.byref(_lib.KvCache(**d))


def rows(d=A, b=4096, t=512, h=64):
    return ctypes.byref(_lib.KvRows(d, b, t, h))


@pytest.mark.parametrize("sequences,tokens,heads", [(65535, 256, 256), (65535, 1, 32770), (4096, 256, 2048)])
def test_attention_refuses_more_rows_than_its_join_takes(lib, sequences, tokens, heads):
    """2^31 query rows and more are refused before the first of the call's two kernels is enqueued: without a GPU, where
    the first CUDA call fails, the answer is that of the check."""
    assert sequences * tokens * heads >= 1 << 31
    got = lib.uzkv_tree_attention(rows(), rows(), A, 0, tokens, heads, None, 0, None, 1.0, cache(sequences=sequences), A, 1 << 60, None)
    assert got == _lib.ERR_ARG
