"""PyTorch front end of the KV-cache operators (``include/uzip_kv.h``): rotary
positions, attention for a tree of drafted tokens, the attention weight that
cached tokens collect, and eviction by that weight into a packed buffer that
the codec then takes (:func:`encode` for bfloat16, :func:`e5m2_encode` for E5M2).

As in the codec's front end, this module marshals arguments and checks what
the C ABI cannot see (devices, types, shapes, strides); a refusal is a
``ValueError`` raised before anything is enqueued, a status of the library an
:class:`UzipError`. Work goes to the current CUDA stream of the tensors'
device and nothing synchronises.

:func:`rotary` and :func:`rotary_backward` take part in autograd. The other
operators have no gradient and refuse inputs whose gradient is being recorded
(``torch.no_grad()`` or ``detach()``), as every operator does where ``out`` is
given.
"""
from __future__ import annotations

import ctypes
import math
import struct
import threading
from dataclasses import dataclass

import torch
from torch.autograd.graph import increment_version

from . import _lib, codec
from ._lib import check, load
from .codec import _at, _sp

# Calls of a few microseconds on the GPU are bound by the host: each call looks
# every attribute up once, and tensors go to the C ABI as packed structures.
_pack_rows = struct.Struct("@Pqqq").pack  # uzkv_rows_t

MAX_HEAD_DIM = 256
MAX_NEW_TOKENS = 256
_DTYPES = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2, torch.float8_e5m2: 3}
_FLOATS = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2}
_LAYOUTS = {"half": 0, "interleaved": 1}


def _tensor(t: torch.Tensor, what: str, dtype, shape=None, device=None) -> torch.Tensor:
    if t.dtype != dtype:
        raise ValueError(f"{what}: expected {dtype}, got {t.dtype}")
    if not t.is_cuda:
        raise ValueError(f"{what}: expected a CUDA tensor")
    if device is not None and t.device != device:
        raise ValueError(f"{what}: on {t.device}, expected {device}")
    if shape is not None and t.shape != shape:
        raise ValueError(f"{what}: shape {tuple(t.shape)}, expected {tuple(shape)}")
    return t


def _dense(t: torch.Tensor, what: str, dtype, shape, device) -> torch.Tensor:
    if not _tensor(t, what, dtype, shape, device).is_contiguous():
        raise ValueError(f"{what}: expected a contiguous tensor")
    return t


def _rows(x: torch.Tensor, what: str) -> bytes:
    """A [sequences, tokens, heads, dim] tensor as the C ABI takes it."""
    sb, st, sh, sd = x.stride()
    if sd != 1 and x.shape[3] != 1:
        raise ValueError(f"{what}: elements of a row must be contiguous")
    return _pack_rows(x.data_ptr(), sb, st, sh)


def _writable(x: torch.Tensor, what: str) -> None:
    """Check an output: no two of its elements in one place."""
    expect = 1
    for n, s in zip(reversed(x.shape), reversed(x.stride())):  # dimensions in their usual order
        if n > 1:
            if s < expect:
                break
            expect += s * (n - 1)
    else:
        return
    expect = 1
    for n, s in sorted(zip(x.shape, x.stride()), key=lambda v: v[1]):
        if n > 1:
            if s < expect:
                raise ValueError(f"{what}: its elements overlap")
            expect += s * (n - 1)


def _overlap(x: torch.Tensor, y: torch.Tensor) -> bool:
    """Whether two tensors share a byte: interleaved views of one buffer need not."""
    x0, y0 = x.data_ptr(), y.data_ptr()
    if y0 < x0:
        x, y, x0, y0 = y, x, y0, x0
    end = 1
    for n, s in zip(x.shape, x.stride()):
        end += (n - 1) * s
    if y0 - x0 >= end * x.element_size() or not x.numel() or not y.numel():
        return False
    # What the last two dimensions span repeats at multiples of g only: heads side by side in one projection.
    g, spans = 0, []
    for t in (x, y):
        size = t.element_size()
        wide = size  # bytes to the end of the last two dimensions
        behind = t.dim() - 2
        for i, (n, s) in enumerate(zip(t.shape, t.stride())):
            if n > 1:
                if i < behind:
                    g = math.gcd(g, s * size)
                else:
                    wide += (n - 1) * s * size
        spans.append(wide)
    if g and spans[0] <= (y0 - x0) % g <= g - spans[1]:
        return False
    # x0 + sum of i s = y0 + sum of j t over x's and y's indexes i, j, strides s, t in bytes and the bytes of an element:
    # one equation in bounded integers, solved from the largest stride down.
    span: dict[int, list[int]] = {}
    for t, sign in ((x, 1), (y, -1)):
        size = t.element_size()
        for n, s in [*((n, s * size) for n, s in zip(t.shape, t.stride())), (size, 1)]:
            if n > 1 and s:
                r = span.setdefault(s, [0, 0])
                r[sign > 0] += sign * (n - 1)
    strides = sorted(span, reverse=True)
    rest = [(0, 0, 0)]  # of the strides behind: least and largest sum, greatest common divisor
    for s in reversed(strides):
        lo, hi, g = rest[-1]
        rest.append((lo + s * span[s][0], hi + s * span[s][1], math.gcd(g, s)))
    rest.reverse()
    budget = 20000

    def reach(k: int, left: int) -> bool:
        nonlocal budget
        budget -= 1
        if budget < 0:
            return True  # undecided: taken as shared
        lo, hi, g = rest[k]
        if not lo <= left <= hi or (left % g if g else left):
            return False
        if k == len(strides):
            return True
        s, (least, most) = strides[k], span[strides[k]]
        lo, hi, _ = rest[k + 1]
        return any(reach(k + 1, left - c * s) for c in range(max(least, -((hi - left) // s)), min(most, (left - lo) // s) + 1))

    return reach(0, y0 - x0)


def _no_gradient(what: str, *tensors) -> None:
    """Refuse tensors whose gradient would be cut without a word."""
    if torch.is_grad_enabled() and any(t is not None and t.requires_grad for t in tensors):
        raise ValueError(f"{what}: has no gradient; call it under torch.no_grad() or on detached tensors")


def _given(out: torch.Tensor, what: str, *apart, in_place=None) -> None:
    """Check a caller's output, which is written past autograd's knowledge: what
    was saved of it is no longer valid. It shares no memory with the ``apart``
    (tensor, name), nor with the one ``in_place``, unless it is that one element
    for element: the call reads them while it writes."""
    _writable(out, what)
    if out.requires_grad:
        _no_gradient(what, out)
    storage = out.untyped_storage().data_ptr()
    for x, name in apart if in_place is None else (in_place, *apart):
        if x.untyped_storage().data_ptr() != storage:
            continue
        if in_place is not None and x is in_place[0] and (out is x or (
                out.data_ptr() == x.data_ptr() and out.shape == x.shape
                and all(n == 1 or s == t for n, s, t in zip(x.shape, out.stride(), x.stride())))):
            continue
        if _overlap(out, x):
            raise ValueError(f"{what}: overlaps {name}")
    increment_version((out,))


# ----------------------------------------------------------------- rotary

@dataclass(frozen=True)
class RotaryPlan:
    """Rates of the pairs of a head, made once and shared by every call."""
    turns: torch.Tensor  # int64 [rotary_dim / 2]: 64-bit fixed-point turns a position
    rotary_dim: int
    layout: str
    magnitude: float

    def __post_init__(self):
        if self.layout not in _LAYOUTS:
            raise ValueError(f"layout {self.layout!r}: expected 'half' or 'interleaved'")
        if self.turns.dtype != torch.int64 or self.turns.shape != (self.rotary_dim // 2,) or not self.turns.is_contiguous():
            raise ValueError("turns: expected a contiguous int64 tensor of rotary_dim / 2")
        # What each call passes on, looked up once.
        object.__setattr__(self, "index", self.turns.get_device())
        object.__setattr__(self, "device", self.turns.device)
        object.__setattr__(self, "args", (self.turns.data_ptr(), self.rotary_dim, _LAYOUTS[self.layout], self.magnitude))


def rotary_rates(rotary_dim: int, base: float = 10000.0, scaling: str = "none", factor: float = 1.0,
                 original_length: int = 0, low: float = 1.0, high: float = 32.0,
                 magnitude: float | None = None) -> tuple[list[float], float]:
    """Radians a position of each pair, and the factor on cosines and sines.

    ``base ** (-2 i / rotary_dim)`` for pair i, and for a context stretched by
    ``factor``: "linear" divides every rate by it; "base" raises the base to
    ``base * factor ** (rotary_dim / (rotary_dim - 2))``, which leaves the
    fastest pair as it is and divides the slowest by ``factor``; "ramp" divides
    the pairs that turn less than ``low`` times over ``original_length``
    positions, leaves those that turn more than ``high`` times, mixes linearly
    between, and scales cosines and sines by ``0.1 ln(factor) + 1``.
    ``magnitude`` replaces the factor that the scaling gives (1 but for "ramp")."""
    rates, given = _rates(rotary_dim, base, scaling, factor, original_length, low, high)
    if magnitude is None:
        return rates, given
    if not (magnitude > 0.0 and math.isfinite(magnitude)):
        raise ValueError("magnitude: expected a positive number")
    return rates, float(magnitude)


def _rates(rotary_dim, base, scaling, factor, original_length, low, high) -> tuple[list[float], float]:
    if rotary_dim < 2 or rotary_dim % 2 or rotary_dim > MAX_HEAD_DIM:
        raise ValueError(f"rotary_dim {rotary_dim}: expected an even number in [2, {MAX_HEAD_DIM}]")
    if not (base > 1.0 and math.isfinite(base) and factor >= 1.0 and math.isfinite(factor)):
        raise ValueError("expected base > 1 and factor >= 1")
    if scaling == "base":
        if rotary_dim == 2:
            raise ValueError("base scaling needs a rotary_dim above 2")
        base = base * factor ** (rotary_dim / (rotary_dim - 2))
    rates = [base ** (-2.0 * i / rotary_dim) for i in range(rotary_dim // 2)]
    if scaling in ("none", "base"):
        return rates, 1.0
    if scaling == "linear":
        return [f / factor for f in rates], 1.0
    if scaling == "ramp":
        if original_length <= 0 or not low < high:
            raise ValueError("ramp scaling needs original_length > 0 and low < high")
        out = []
        for f in rates:
            turns = original_length * f / (2 * math.pi)
            g = min(1.0, max(0.0, (turns - low) / (high - low)))
            out.append(f * (g + (1.0 - g) / factor))
        return out, 0.1 * math.log(factor) + 1.0
    raise ValueError(f"scaling {scaling!r}: expected 'none', 'linear', 'base' or 'ramp'")


def rotary_plan(rotary_dim: int, base: float = 10000.0, layout: str = "half", scaling: str = "none",
                factor: float = 1.0, original_length: int = 0, low: float = 1.0, high: float = 32.0,
                device="cuda", magnitude: float | None = None) -> RotaryPlan:
    """The plan of :func:`rotary` and :func:`rotary_append`; see :func:`rotary_rates`
    for the scalings and ``magnitude``. ``layout``: "half" turns elements i and i + rotary_dim / 2
    together, "interleaved" 2 i and 2 i + 1."""
    rates, magnitude = rotary_rates(rotary_dim, base, scaling, factor, original_length, low, high, magnitude)
    turns = [int(round(f / (2 * math.pi) * 2.0 ** 64)) for f in rates]
    turns = torch.tensor([v - (1 << 64) if v >= 1 << 63 else v for v in turns], dtype=torch.int64, device=device)
    return RotaryPlan(turns, rotary_dim, layout, magnitude)


def _positions(positions, b, t, index) -> int:
    """Check int32 positions [b, t]; the stride between their rows."""
    shape = positions.shape
    if positions.dtype is not torch.int32 or len(shape) != 2 or shape[0] != b or shape[1] != t or positions.get_device() != index:
        raise ValueError(f"positions: expected int32 of the tensor's {b} x {t} tokens on its device")
    sb, st = positions.stride()
    if st != 1 and t > 1:
        raise ValueError("positions: expected contiguous rows")
    return sb


class _Rotary(torch.autograd.Function):
    """The turn (or, backward, the turn back), whose gradient is the other one."""

    @staticmethod
    def forward(ctx, x, positions, plan, backward):
        ctx.save_for_backward(positions)
        ctx.plan, ctx.backward_ = plan, backward
        return _rotate(x, positions, plan, None, backward)

    @staticmethod
    def backward(ctx, grad):
        (positions,) = ctx.saved_tensors
        if grad.stride(-1) != 1:  # a sum's gradient is one element expanded
            grad = grad.contiguous()
        return _rotate(grad, positions, ctx.plan, None, 1 - ctx.backward_), None, None, None


def _rotate(x, positions, plan, out, backward):
    if x.requires_grad and torch.is_grad_enabled():
        if out is not None:
            _no_gradient("out", x)
        return _Rotary.apply(x, positions, plan, backward)
    kind, shape, index = _FLOATS.get(x.dtype), x.shape, x.get_device()
    if kind is None:
        raise ValueError(f"expected bfloat16, float16 or float32 values, got {x.dtype}")
    if len(shape) == 3:  # [tokens, heads, dim]
        if positions.dim() != 1:
            raise ValueError("positions: expected one for each token")
        got = _rotate(x[None], positions[None], plan, None if out is None else out[None], backward)
        return got[0] if out is None else out
    if len(shape) != 4 or index < 0:
        raise ValueError("expected a CUDA tensor [tokens, heads, dim] or [sequences, tokens, heads, dim]")
    if plan.index != index:
        raise ValueError("plan: on another device")
    b, t, heads, d = shape
    step = _positions(positions, b, t, index)
    empty = b * t * heads * d == 0
    rx = None if empty else _rows(x, "x")  # no rule for the strides of nothing
    if out is None:
        out = torch.empty((b, t, heads, d), dtype=x.dtype, device=plan.device)
        ro = _pack_rows(out.data_ptr(), t * heads * d, heads * d, d)
    else:
        _given(_tensor(out, "out", x.dtype, shape, x.device), "out", in_place=(x, "x"))
        ro = _rows(out, "out")
    if empty:
        return out
    turns, rotary_dim, layout, magnitude = plan.args
    rc = _at(index, load().uzkv_rotary)(
        rx, ro, kind, b, t, heads, d, positions.data_ptr(), step, turns, rotary_dim, layout, magnitude, backward,
        _sp(index))
    if rc:
        check(rc, "uzkv_rotary")
    return out


def rotary(x: torch.Tensor, positions: torch.Tensor, plan: RotaryPlan,
           out: torch.Tensor | None = None) -> torch.Tensor:
    """Turn the pairs of each head of ``x`` ([tokens, heads, dim] or
    [sequences, tokens, heads, dim], bfloat16, float16 or float32, rows
    contiguous) by its token's position (int32). Elements past the plan's
    rotary_dim are copied. ``out`` may be ``x`` (or lie apart from it). Differentiable in ``x`` where
    ``out`` is not given."""
    return _rotate(x, positions, plan, out, 0)


def rotary_backward(grad: torch.Tensor, positions: torch.Tensor, plan: RotaryPlan,
                    out: torch.Tensor | None = None) -> torch.Tensor:
    """Gradient of :func:`rotary`'s input from that of its output: the same
    turn, backwards. What autograd calls for :func:`rotary`; for training loops
    that keep their own tape. Differentiable like it."""
    return _rotate(grad, positions, plan, out, 1)


# ------------------------------------------------------------------ cache

class KVCache:
    """One layer's cache, as every operator here takes it; made once and kept.

    ``k``, ``v``: pools of pages [pages, kv heads, page tokens, head dim] of
    bfloat16, float16 or float8_e5m2 (views are fine: rows contiguous, other
    strides multiples of 16 bytes). ``page_table`` int32 [sequences, pages of a
    sequence], read for tokens in use only. ``lengths`` int32 [sequences]: tokens
    of each sequence before the new ones of a call; the tensor is read on the
    device by each call, so advance it in place (``cache.lengths += n``). Every
    call passes on the addresses taken here, so the attributes cannot be set to
    other tensors, nor may a tensor's storage be exchanged: make a new KVCache.
    ``status``: None or one int32 CUDA element that a call sets to 5 (corrupt)
    when a length or page number is out of range (6 if a bounded wait inside a
    kernel ran out; never cleared). A contiguous cache [sequences, heads, tokens,
    dim] is the pool of whole-sequence pages with
    ``page_table = arange(sequences)[:, None]``. A batch of no sequences gives
    empty results."""

    def __init__(self, k: torch.Tensor, v: torch.Tensor, page_table: torch.Tensor, lengths: torch.Tensor,
                 status: torch.Tensor | None = None):
        if k.dim() != 4 or k.dtype not in _DTYPES or k.dtype == torch.float32:
            raise ValueError("k: expected [pages, kv heads, page tokens, head dim] of bfloat16, float16 or float8_e5m2")
        _tensor(k, "k", k.dtype)
        _tensor(v, "v", k.dtype, k.shape, k.device)
        if page_table.dim() != 2:
            raise ValueError("page_table: expected [sequences, pages of a sequence]")
        _tensor(page_table, "page_table", torch.int32, None, k.device)
        if page_table.shape[1] > 1 and page_table.stride(1) != 1:
            raise ValueError("page_table: expected contiguous rows")
        _dense(lengths, "lengths", torch.int32, page_table.shape[:1], k.device)
        if status is not None:
            _dense(status, "status", torch.int32, torch.Size([1]), k.device)
        for t, what in ((k, "k"), (v, "v")):
            _writable(t, what)
            if t.requires_grad:
                raise ValueError(f"{what}: a cache is written past autograd's knowledge; give detached tensors")
            if t.shape[3] > 1 and t.stride(3) != 1:
                raise ValueError(f"{what}: elements of a row must be contiguous")
        self.k, self.v, self.page_table, self.lengths, self.status = k, v, page_table, lengths, status
        self.device, self.dtype, self.index = k.device, k.dtype, k.get_device()
        self.takes = (torch.bfloat16, torch.float16) if k.dtype == torch.float8_e5m2 else (k.dtype,)
        self.sequences, self.kv_heads, self.head_dim = page_table.shape[0], k.shape[1], k.shape[3]
        self.page_tokens = k.shape[2]
        self.capacity = page_table.shape[1] * k.shape[2]
        self._c = _lib.KvCache(
            k.data_ptr(), v.data_ptr(), *k.stride()[:3], *v.stride()[:3], page_table.data_ptr(), page_table.stride(0),
            lengths.data_ptr(), status.data_ptr() if status is not None else None, k.shape[0], k.shape[1], k.shape[2],
            k.shape[3], page_table.shape[0], page_table.shape[1], _DTYPES[k.dtype], 0)
        self._ref = ctypes.byref(self._c)
        self._workspace_bytes: dict[tuple[int, int], int] = {}  # by (tokens, heads)

    def __setattr__(self, name, value):
        # The same object again is what `cache.lengths += n` assigns.
        if self.__dict__.get(name, value) is not value:
            raise AttributeError(f"{name}: a cache keeps its tensors; change them in place or make a new KVCache")
        self.__dict__[name] = value

    def __delattr__(self, name):
        raise AttributeError(f"{name}: a cache keeps its tensors")


def _new_rows(x: torch.Tensor, what: str, cache: KVCache, heads: int | None = None) -> bytes:
    """Check new tokens' rows [sequences, tokens, heads, head dim] of a cache."""
    shape = x.shape
    if len(shape) != 4 or shape[0] != cache.sequences or shape[3] != cache.head_dim or x.get_device() != cache.index \
            or (heads is not None and shape[2] != heads):
        raise ValueError(f"{what}: expected [{cache.sequences}, tokens, {heads or 'heads'}, {cache.head_dim}] "
                         f"on {cache.device}, got {tuple(shape)} on {x.device}")
    if x.dtype not in cache.takes:
        raise ValueError(f"{what}: {x.dtype} does not go with a cache of {cache.dtype}")
    sb, st, sh, sd = x.stride()
    if sd != 1 and shape[3] != 1:
        raise ValueError(f"{what}: elements of a row must be contiguous")
    return _pack_rows(x.data_ptr(), sb, st, sh)


def _new_out(out: torch.Tensor | None, q: torch.Tensor, b: int, t: int, heads: int, d: int, device, *apart):
    """The output of q's shape (a new one where None, else q or apart from it and from ``apart``), and its rows."""
    if out is None:
        out = torch.empty((b, t, heads, d), dtype=q.dtype, device=device)
        return out, _pack_rows(out.data_ptr(), t * heads * d, heads * d, d)
    _given(_tensor(out, "out", q.dtype, q.shape, device), "out", *apart, in_place=(q, "q"))
    return out, _rows(out, "out")


def _counts(counts, cache):
    if counts is None:
        return None
    if counts.dtype != torch.int32 or counts.shape != (cache.sequences,) or counts.get_device() != cache.index \
            or not counts.is_contiguous():
        raise ValueError(f"counts: expected a contiguous int32 tensor of {cache.sequences} on {cache.device}")
    return counts.data_ptr()


def rotary_append(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, positions: torch.Tensor, plan: RotaryPlan,
                  cache: KVCache, counts: torch.Tensor | None = None, out: torch.Tensor | None = None) -> torch.Tensor:
    """Rotate the queries and keys of new tokens, store keys and values in the
    cache at slots lengths .. lengths + counts - 1 (rounded once to its type) and
    return the rotated queries, in one launch. ``q`` [sequences, tokens, query
    heads, dim], ``k`` and ``v`` [sequences, tokens, kv heads, dim] (views of one
    projection are fine), ``positions`` int32 [sequences, tokens]. Tokens at or
    past ``counts`` give zero queries and are not stored. ``out`` may be ``q``.
    Advancing ``cache.lengths`` is the caller's, once the tokens are accepted."""
    kv_heads, index = cache.kv_heads, cache.index
    if q.requires_grad or k.requires_grad or v.requires_grad:
        _no_gradient("rotary_append", q, k, v)
    rq, rk, rv = _new_rows(q, "q", cache), _new_rows(k, "k", cache, kv_heads), _new_rows(v, "v", cache, kv_heads)
    b, t, heads, d = q.shape
    dtype = q.dtype
    if k.shape[1] != t or v.shape[1] != t or k.dtype is not dtype or v.dtype is not dtype:
        raise ValueError("k, v: type or tokens differ from q's")
    if plan.index != index:
        raise ValueError("plan: on another device")
    step = _positions(positions, b, t, index)
    if heads == 0:
        raise ValueError("q: no heads")
    out, ro = _new_out(out, q, b, t, heads, d, cache.device, (k, "k"), (v, "v"))
    if b * t == 0:
        return out
    turns, rotary_dim, layout, magnitude = plan.args
    rc = _at(index, load().uzkv_rotary_append)(
        rq, rk, rv, ro, _FLOATS[dtype], t, heads, positions.data_ptr(), step, turns, rotary_dim, layout, magnitude,
        _counts(counts, cache), cache._ref, _sp(index))
    if rc:
        check(rc, "uzkv_rotary_append")
    return out


# -------------------------------------------------------------- attention

def tree_mask(parents, device="cuda") -> torch.Tensor:
    """Mask rows of drafted trees: ``parents[b][t]`` is the node that token t of
    sequence b continues, or -1 for one that continues the cache; a parent comes
    before its child. Returns int64 [sequences, tokens, ceil(tokens / 64)]: bit u
    of row t is set where u is t or an ancestor of t. The host does not wait for
    the copy to ``device``, which the current stream makes. Not under a graph's
    capture, whose replays would copy from memory that is gone."""
    rows = [[int(u) for u in row] for row in parents]
    t = len(rows[0]) if rows else 0
    if not 1 <= t <= MAX_NEW_TOKENS or any(len(r) != t for r in rows):
        raise ValueError(f"parents: expected rows of one length in [1, {MAX_NEW_TOKENS}]")
    words = -(-t // 64)
    out = []
    for row in rows:
        seen: list[int] = []
        for i, u in enumerate(row):
            if not -1 <= u < i:
                raise ValueError(f"parents: node {i} has parent {u}")
            seen.append((seen[u] if u >= 0 else 0) | 1 << i)
        out.append([[(w - (1 << 64) if w >= 1 << 63 else w)
                     for w in ((s >> 64 * j) & ((1 << 64) - 1) for j in range(words))] for s in seen])
    mask = torch.tensor(out, dtype=torch.int64)
    device = torch.device(device)
    if device.type != "cuda":
        return mask.to(device)
    if _capturing(codec._current_device() if device.index is None else device.index):
        raise ValueError("tree_mask: a replay would not see the tree; make masks before the capture")
    return mask.pin_memory().to(device, non_blocking=True)  # from pageable memory the host would wait for the stream


def _mask(mask, cache, t):
    """(address, words between sequences) of a mask."""
    words = -(-t // 64)
    if mask.dim() != 3 or mask.shape[0] not in (1, cache.sequences) or mask.shape[1:] != (t, words):
        raise ValueError(f"mask: expected [{cache.sequences} or 1, {t}, {words}], got {tuple(mask.shape)}")
    if mask.dtype != torch.int64 or mask.get_device() != cache.index or not mask.is_contiguous():
        raise ValueError(f"mask: expected a contiguous int64 tensor on {cache.device}")
    return mask.data_ptr(), 0 if mask.shape[0] == 1 else t * words


def _query(q: torch.Tensor, cache: KVCache):
    """Check queries of new tokens; their rows and shape."""
    if q.requires_grad:
        _no_gradient("q", q)
    rows = _new_rows(q, "q", cache)
    b, t, heads, d = q.shape
    if not 1 <= t <= MAX_NEW_TOKENS:
        raise ValueError(f"q: {t} new tokens, expected 1 to {MAX_NEW_TOKENS}")
    if heads == 0 or heads % cache.kv_heads:
        raise ValueError(f"q: {heads} heads over {cache.kv_heads} kv heads")
    return rows, b, t, heads, d


def _floats(x: torch.Tensor, what: str, shape, cache: KVCache) -> int:
    """Address of a contiguous float32 tensor of the given shape."""
    if x.dtype != torch.float32 or x.shape != shape or x.get_device() != cache.index or not x.is_contiguous():
        raise ValueError(f"{what}: expected contiguous float32 {tuple(shape)} on {cache.device}")
    return x.data_ptr()


def tree_attention_workspace_bytes(cache: KVCache, tokens: int, heads: int) -> int:
    size = cache._workspace_bytes.get((tokens, heads))
    if size is None:
        size = int(load().uzkv_tree_attention_workspace_bytes(cache.sequences, tokens, heads, cache.kv_heads,
                                                              cache.head_dim))
        cache._workspace_bytes[tokens, heads] = size
    return size


_scratch = threading.local()


def _capturing(index: int) -> bool:
    """Whether the current stream of device ``index`` is being captured in a graph."""
    if index == codec._current_device():
        return torch.cuda.is_current_stream_capturing()
    with torch.cuda.device(index):
        return torch.cuda.is_current_stream_capturing()


def _workspace(cache: KVCache, size: int) -> torch.Tensor:
    """Scratch of at least ``size`` bytes for a call on the current stream: one
    buffer a host thread and stream, which its calls use one after the other. A
    call under graph capture gets its own, which the graph then holds."""
    if _capturing(cache.index):
        return torch.empty(size, dtype=torch.uint8, device=cache.device)
    buffers = _scratch.__dict__
    key = (cache.index, _sp(cache.index))
    buffer = buffers.get(key)
    if buffer is None or buffer.numel() < size:
        buffer = buffers[key] = torch.empty(size, dtype=torch.uint8, device=cache.device)
    return buffer


def tree_attention(q: torch.Tensor, cache: KVCache, mask: torch.Tensor | None = None,
                   counts: torch.Tensor | None = None, scale: float | None = None, out: torch.Tensor | None = None,
                   lse: torch.Tensor | None = None, workspace: torch.Tensor | None = None):
    """Attention of new tokens over the cache that already holds their keys and
    values (:func:`rotary_append`). ``q`` [sequences, tokens, query heads, dim],
    1 to 256 tokens (``out`` may be ``q``); token t sees the first lengths slots and the new tokens of
    its mask row (:func:`tree_mask`; one tree for all when the mask has one
    sequence; None: a chain, each token and those before it). Returns ``(out,
    lse)``: the output, and the float32 log-sum-exp [sequences, tokens, heads].
    Rows that see nothing, and tokens at or past ``counts``, give 0 and -inf.
    ``workspace``: :func:`tree_attention_workspace_bytes` of uint8 that no call
    on another stream uses meanwhile; None takes a buffer that is kept for the
    calling thread's work on this stream (up to 43 MB)."""
    rq, b, t, heads, d = _query(q, cache)
    address, stride = _mask(mask, cache, t) if mask is not None else (None, 0)
    out, ro = _new_out(out, q, b, t, heads, d, cache.device)
    if lse is None:
        lse = torch.empty((b, t, heads), dtype=torch.float32, device=cache.device)
        at_lse = lse.data_ptr()
    else:
        at_lse = _floats(lse, "lse", (b, t, heads), cache)
        if lse.requires_grad:
            _no_gradient("lse", lse)
        increment_version((lse,))
    if b == 0:
        return out, lse
    if workspace is None:
        workspace = _workspace(cache, tree_attention_workspace_bytes(cache, t, heads))
    elif not _tensor(workspace, "workspace", torch.uint8, None, cache.device).is_contiguous():
        raise ValueError("workspace: expected a contiguous tensor")
    rc = _at(cache.index, load().uzkv_tree_attention)(
        rq, ro, at_lse, _FLOATS[q.dtype], t, heads, address, stride, _counts(counts, cache),
        d ** -0.5 if scale is None else scale, cache._ref, workspace.data_ptr(), workspace.numel(), _sp(cache.index))
    if rc:
        check(rc, "uzkv_tree_attention")
    return out, lse


def attention_mass(q: torch.Tensor, cache: KVCache, lse: torch.Tensor, mask: torch.Tensor | None = None,
                   counts: torch.Tensor | None = None, weights: torch.Tensor | None = None,
                   mass: torch.Tensor | None = None, decay: float = 1.0, scale: float | None = None,
                   out: torch.Tensor | None = None) -> torch.Tensor:
    """The attention weight that each cached token collects: float32 [sequences,
    kv heads, slots], ``decay * mass`` for the tokens already in the cache plus,
    over the group's heads and the new tokens that see it, ``weights[b, t] *
    exp(score - lse)``; 0 for slots not in use. ``q``, ``mask``, ``counts`` and
    ``scale`` as for the :func:`tree_attention` that gave ``lse``; ``weights``
    float32 [sequences, tokens] (1 for accepted tokens, 0 for the others; None:
    ones). ``out`` may be ``mass``; a ``mass`` whose rows lie otherwise than
    ``out``'s is first copied there. ``out``'s width (default: the cache's capacity) says
    how many slots are weighed."""
    rq, b, t, heads, d = _query(q, cache)
    address, stride = _mask(mask, cache, t) if mask is not None else (None, 0)
    at_lse = _floats(lse, "lse", (b, t, heads), cache)
    at_weights = _floats(weights, "weights", (b, t), cache) if weights is not None else None
    if lse.requires_grad or (weights is not None and weights.requires_grad) or (mass is not None and mass.requires_grad):
        _no_gradient("attention_mass", lse, weights, mass)
    kv_heads = cache.kv_heads
    if out is None:
        out = torch.empty(mass.shape if mass is not None else (b, kv_heads, cache.capacity), dtype=torch.float32,
                          device=cache.device)
    else:
        reads = [(lse, "lse")] if weights is None else [(lse, "lse"), (weights, "weights")]
        _given(_tensor(out, "out", torch.float32, None, cache.device), "out", *reads,
               in_place=None if mass is None else (mass, "mass"))
    shape = out.shape
    if len(shape) != 3 or shape[0] != b or shape[1] != kv_heads or not 1 <= shape[2] <= cache.capacity:
        raise ValueError(f"out: expected [{b}, {kv_heads}, 1 to {cache.capacity}], got {tuple(shape)}")
    sb, sh, sn = out.stride()
    if shape[2] > 1 and sn != 1:
        raise ValueError("out: expected contiguous rows")
    at_mass = None
    if mass is not None:
        if mass.dtype != torch.float32 or mass.get_device() != cache.index or mass.shape != shape:
            raise ValueError(f"mass: expected float32 {tuple(shape)} on {cache.device}")
        if mass.stride() != (sb, sh, sn) and any(n > 1 and s != t for n, s, t in zip(shape, mass.stride(), (sb, sh, sn))):
            mass = out.copy_(mass)  # the kernel takes both with the same strides; they may be one
        at_mass = mass.data_ptr()
    if b == 0:
        return out
    rc = _at(cache.index, load().uzkv_attention_mass)(
        rq, at_lse, _FLOATS[q.dtype], t, heads, address, stride, _counts(counts, cache), at_weights,
        d ** -0.5 if scale is None else scale, cache._ref, at_mass, decay, out.data_ptr(), sb, sh, shape[2],
        _sp(cache.index))
    if rc:
        check(rc, "uzkv_attention_mass")
    return out


# --------------------------------------------------------------- eviction

@dataclass
class Packed:
    """What :func:`evict` keeps: ``k``, ``v`` [sequences, kv heads, keep, dim],
    ``mass`` float32 and ``kept`` int32 [sequences, kv heads, keep] (slots in
    ascending order), ``lengths`` int32 [sequences]. Rows past a sequence's length
    are zero, -1 in ``kept``."""
    k: torch.Tensor
    v: torch.Tensor
    mass: torch.Tensor
    kept: torch.Tensor
    lengths: torch.Tensor


def evict(cache: KVCache, mass: torch.Tensor, keep: int, sink: int = 0, recent: int = 0,
          out_k: torch.Tensor | None = None, out_v: torch.Tensor | None = None) -> Packed:
    """Keep ``keep`` tokens of each sequence and head and pack them: the first
    ``sink``, the last ``recent`` and those of the largest ``mass`` (float32
    [sequences, kv heads, slots]; equal masses: the lowest slot first). A sequence
    of at most ``keep`` tokens keeps them all. ``out_k`` and ``out_v`` default to new
    contiguous tensors, ready for :func:`encode` (bfloat16) or :func:`e5m2_encode`;
    float16 has no format of its own, ``encode`` takes its bits but its codebook is
    for bfloat16's exponent field. Given ones may be the halves of one buffer or
    views with room behind for tokens to come, but no part of the cache."""
    b, heads, d = cache.sequences, cache.kv_heads, cache.head_dim
    shape = mass.shape
    if mass.dtype is not torch.float32 or mass.get_device() != cache.index or len(shape) != 3 or shape[0] != b \
            or shape[1] != heads or shape[2] < 1:
        raise ValueError(f"mass: expected float32 [{b}, {heads}, slots] on {cache.device}, got {mass.dtype} "
                         f"{tuple(shape)} on {mass.device}")
    sb, sh, sn = mass.stride()
    if shape[2] > 1 and sn != 1:
        raise ValueError("mass: expected contiguous rows")
    if mass.requires_grad:
        _no_gradient("evict", mass)
    if keep < 1 or sink < 0 or recent < 0 or sink + recent > keep:
        raise ValueError("expected keep >= 1 and 0 <= sink + recent <= keep")
    device = cache.device
    if out_k is None and out_v is None:
        out_k, out_v = (torch.empty((b, heads, keep, d), dtype=cache.dtype, device=device) for _ in range(2))
        rk, rv = (_pack_rows(x.data_ptr(), heads * keep * d, keep * d, d) for x in (out_k, out_v))
    elif out_k is None or out_v is None:
        raise ValueError("give both out_k and out_v or neither")
    else:
        pools = (cache.k, "the cache"), (cache.v, "the cache")
        for x, what in ((out_k, "out_k"), (out_v, "out_v")):
            _tensor(x, what, cache.dtype, (b, heads, keep, d), device)
        _given(out_k, "out_k", *pools, (out_v, "out_v"))
        _given(out_v, "out_v", *pools)
        rk, rv = _rows(out_k, "out_k"), _rows(out_v, "out_v")
    kept = torch.empty((b, heads, keep), dtype=torch.int32, device=device)
    mass_out = torch.empty((b, heads, keep), dtype=torch.float32, device=device)
    lengths = torch.empty((b,), dtype=torch.int32, device=device)
    if b == 0:
        return Packed(out_k, out_v, mass_out, kept, lengths)
    rc = _at(cache.index, load().uzkv_evict)(
        cache._ref, mass.data_ptr(), sb, sh, shape[2], keep, sink, recent, rk, rv, kept.data_ptr(), mass_out.data_ptr(),
        lengths.data_ptr(), _sp(cache.index))
    if rc:
        check(rc, "uzkv_evict")
    return Packed(out_k, out_v, mass_out, kept, lengths)


__all__ = ["KVCache", "MAX_HEAD_DIM", "MAX_NEW_TOKENS", "Packed", "RotaryPlan", "attention_mass", "evict", "rotary",
           "rotary_append", "rotary_backward", "rotary_plan", "rotary_rates", "tree_attention",
           "tree_attention_workspace_bytes", "tree_mask"]
