"""uzip: fixed-length lossless BF16 exponent codec (SplitZip) for NVIDIA GB300.

The codec itself is ``libuzip.so`` (hand-written CUDA for sm_103a, C ABI in
``include/uzip.h``), which also holds the operators on a KV cache (``kv``, C
ABI in ``include/uzip_kv.h``); this package holds its build script, the ctypes / PyTorch
front end and the seeded synthetic workloads. Importing the package does not
load the library; the first codec call does, and fails loudly if it is
missing.
"""
from .codec import (CODEBOOK_BYTES, HEADER_BYTES, UzipError, calibrate, codebook_exps, codebook_from_exps,
                    codebook_histogram, compressed_size, decode, e5m2_calibrate, e5m2_compressed_size,
                    e5m2_decode, e5m2_encode, encode, encode_dynamic, load, make_sentinel, max_compressed_size,
                    new_codebook, roundtrip_ok, sentinel_compressed_size, sentinel_decode, sentinel_encode,
                    stream_copy, stream_info, workspace_bytes)
from .kv import (KVCache, Packed, RotaryPlan, attention_mass, evict, rotary, rotary_append, rotary_backward,
                 rotary_plan, rotary_rates, tree_attention, tree_attention_workspace_bytes, tree_mask)

__all__ = [
    "CODEBOOK_BYTES", "HEADER_BYTES", "UzipError", "calibrate", "codebook_exps", "codebook_from_exps",
    "codebook_histogram", "compressed_size", "decode", "e5m2_calibrate", "e5m2_compressed_size", "e5m2_decode",
    "e5m2_encode", "encode", "encode_dynamic", "load", "make_sentinel", "max_compressed_size",
    "sentinel_compressed_size", "sentinel_decode", "sentinel_encode",
    "new_codebook", "roundtrip_ok", "stream_copy", "stream_info", "workspace_bytes",
    "KVCache", "Packed", "RotaryPlan", "attention_mass", "evict", "rotary", "rotary_append", "rotary_backward",
    "rotary_plan", "rotary_rates", "tree_attention", "tree_attention_workspace_bytes", "tree_mask",
]
