"""Decoding around a paged key-value cache: Python binding of the qmv_kv_* and
qmv_beam_* entry points of ``include/qmv.h`` (argument checks and marshalling
only).

A cache is given as its two pools, keys and values, each either

* a bf16 tensor [pages, heads, page_size, head_dim], or
* ``(codes, scales, biases)`` in ``qmv_pack``'s format: int32 [pages, heads,
  page_size, head_dim*bits/32] and bf16 [.., head_dim/group_size], with
  ``bits`` 8 or 4.

Any strides will do as long as a row is contiguous and all tensors of a cache
have the same strides in rows, so [pages, page_size, heads, head_dim] memory is
passed as its ``transpose(1, 2)`` view.  ``block_tables`` is int32 [B, columns]:
slot t of sequence b lies in page ``block_tables[b, t // page_size]``.

With ``stream`` a call's kernels run there, and what it allocates itself
(workspace, results) belongs to that stream, as under ``torch.cuda.stream``.
"""
from __future__ import annotations

import contextlib
import ctypes
import functools
import struct

import torch

from . import QMV_OUT_BF16, QMV_OUT_F32, _call, _out_code

_P, _I64, _I = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int
_SZ = ctypes.c_size_t
_CACHE = struct.Struct("=6Q4q5i4x")   # qmv_kv_cache; travels as the bytes it packs to
SIGNATURES = {
    "qmv_kv_append": [_P, _I64, _I64, _P, _I64, _I64, _P, _P, _I64, _I64, _I64, _P, _P, _I64, _P, _P, _P, _I64, _I64,
                      _I64, _P],
    "qmv_kv_attend_workspace_bytes": [_P, _I64, _I64, _I, _I, _I64, _P],
    "qmv_kv_attend": [_P, _I64, _I64, _P, _P, _I64, _I64, _P, _I64, _I, ctypes.c_float, _P, _I64, _I64, _I64, _P, _P,
                      _I64, _I64, _I64, _P, _P, _I64, _I, _P, _SZ, _P],
    "qmv_kv_evict_workspace_bytes": [_I64, _I, _I64, _I64, _P],
    "qmv_kv_evict": [_P, _P, _I64, _I64, _P, _I64, _P, _P, _I64, _I64, _I64, _P, _I64, _I64, _P, _P, _P, _P, _SZ, _P],
    "qmv_beam_select_workspace_bytes": [_I64, _I64, _I64, _I, _P],
    "qmv_beam_select": [_P, _I, _I64, _P, _I64, _I64, _I64, _I, _P, _P, _P, _P, _SZ, _P],
    "qmv_beam_reorder": [_P, _P, _P, _I64, _I64, _I64, _P, _I64, _I64, _P, _P, _P, _P],
}
_I32, _F32, _BF16, _U8 = torch.int32, torch.float32, torch.bfloat16, torch.uint8


# ----------------------------------------------------------------- helpers
# A decode loop makes the same calls with the same shapes at every step, so
# everything that follows from shapes, strides, types and devices (the checks,
# the sizes) is worked out once per combination: the _plan functions see these
# plain values only, never a tensor or an address.
_plan = functools.lru_cache(maxsize=1024)


def _spec(t, name):
    if t is None:
        return None
    if not isinstance(t, torch.Tensor):
        raise ValueError(f"{name} must be a device tensor")
    return t.shape, t.stride(), t.dtype, t.device


def _pool_spec(pool, name):
    if isinstance(pool, torch.Tensor):
        return _spec(pool, name)
    if not isinstance(pool, (tuple, list)) or len(pool) != 3:
        raise ValueError("k_cache and v_cache must both be tensors, or both (codes, scales, biases)")
    return tuple(_spec(t, f"{name} {part}") for part, t in zip(("codes", "scales", "biases"), pool))


def _dev(spec, dtype, name, dim=None):
    """A device tensor of this type and number of axes, its last one contiguous."""
    if spec is None:
        raise ValueError(f"{name} is required")
    shape, stride, has, device = spec
    if device.type != "cuda":
        raise ValueError(f"{name} must be a device tensor")
    if has != dtype:
        raise ValueError(f"{name} must be {dtype}, got {has}")
    if dim is not None and len(shape) != dim:
        raise ValueError(f"{name} must have {dim} axes, got {len(shape)}")
    if len(shape) and stride[-1] != 1 and shape[-1] > 1:
        raise ValueError(f"{name} must be contiguous along its last axis")
    return shape


def _whole(spec, dtype, name, shape):
    """A contiguous device tensor of exactly this shape."""
    _dev(spec, dtype, name)
    if tuple(spec[0]) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(spec[0])}")
    step = 1
    for size, stride in zip(reversed(spec[0]), reversed(spec[1])):
        if size > 1 and stride != step:
            raise ValueError(f"{name} must be contiguous")
        step *= size


def _slots(spec):
    """(strides of axes 0 and 1, S) of a [B, heads, S] array; an axis of size one
    has no stride."""
    shape, stride = spec[0], spec[1]
    return stride[0] if shape[0] > 1 else 0, stride[1] if shape[1] > 1 else 0, shape[2]


def _workspace_ok(spec):
    if spec is not None:
        if spec[3].type != "cuda":
            raise ValueError("workspace must be a contiguous device tensor")
        _whole(spec, spec[2], "workspace", spec[0])


def _one_device(first, *others):
    for spec in others:
        if spec is not None and spec[3] != first[3]:
            raise ValueError("all tensors must be on one device")


def _row_strides(spec, name):
    """The strides of axes 0-2 in rows of shape[3] values."""
    shape, strides = spec[0], spec[1]
    out = []
    for size, stride in zip(shape[:3], strides[:3]):
        if size > 1 and (stride % shape[3] or stride <= 0):
            raise ValueError(f"{name}: strides must be positive multiples of a row's {shape[3]} values")
        out.append(max(1, stride // shape[3]) if size > 1 else 1)
    return tuple(out)


def _cache_dims(k, v, group_size, bits):
    """-> (pages, page, head and slot strides, heads, page size, head_dim, bits, group size)."""
    if len(k) != len(v) or isinstance(k[0], torch.Size) != isinstance(v[0], torch.Size):
        raise ValueError("k_cache and v_cache must both be tensors, or both (codes, scales, biases)")
    if isinstance(k[0], torch.Size):
        _dev(k, _BF16, "k_cache", 4)
        _dev(v, _BF16, "v_cache", 4)
        _one_device(k, v)
        if k[0] != v[0]:
            raise ValueError("k_cache and v_cache must have one shape")
        rows = _row_strides(k, "k_cache")
        if rows != _row_strides(v, "v_cache"):
            raise ValueError("k_cache and v_cache must have the same strides")
        pages, heads, page, D = k[0]
        return (pages, *rows, heads, page, D, 16, 0)
    if bits not in (8, 4) or group_size not in (32, 64, 128):
        raise ValueError("a cache of codes has bits 8 or 4 and group_size 32, 64 or 128")
    shape = _dev(k[0], _I32, "k_cache codes", 4)
    D = shape[3] * 32 // bits
    rows = None
    for name, pool in (("k_cache", k), ("v_cache", v)):
        for part, t in zip(("codes", "scales", "biases"), pool):
            _dev(t, _I32 if part == "codes" else _BF16, f"{name} {part}", 4)
            _one_device(k[0], t)
            width = shape[3] if part == "codes" else D // group_size
            if t[0][:3] != shape[:3] or t[0][3] != width or D % group_size:
                raise ValueError(f"{name} {part}: shape {tuple(t[0])} does not fit codes of shape {tuple(shape)} with "
                                 f"bits={bits}, group_size={group_size}")
            r = _row_strides(t, f"{name} {part}")
            if rows is not None and r != rows:
                raise ValueError("all tensors of a cache must have the same strides in rows")
            rows = r
    pages, heads, page, _ = shape
    return (pages, *rows, heads, page, D, bits, group_size)


def _first(pool):
    """The spec of a pool's rows."""
    return pool if isinstance(pool[0], torch.Size) else pool[0]


def _cache(k, v, dims):
    if isinstance(k, torch.Tensor):
        return _CACHE.pack(k.data_ptr(), v.data_ptr(), 0, 0, 0, 0, *dims)
    return _CACHE.pack(k[0].data_ptr(), v[0].data_ptr(), k[1].data_ptr(), k[2].data_ptr(), v[1].data_ptr(),
                       v[2].data_ptr(), *dims)


@_plan
def _bytes(name, *args):
    out = _SZ(0)
    _call(name, *args, ctypes.byref(out))
    return int(out.value)


def _attend_bytes(dims, B, cols, group, weights, max_length):
    # pointers and strides take no part in the size, but have to be valid
    return _bytes("qmv_kv_attend_workspace_bytes", _CACHE.pack(*(16,) * 6, dims[0], 1, 1, 1, *dims[4:]), B, cols, group,
                  weights, max_length)


def _stream(stream, device):
    # the raw handle of the current stream, without a Stream object around it
    return torch._C._cuda_getCurrentRawStream(device.index) if stream is None else stream.cuda_stream


_HERE = contextlib.nullcontext()


def _owner(stream):
    """Where a call's own allocations have to be made: memory of the current
    stream's pool may be in use there, and is handed out there again as soon as
    a workspace is dropped, whatever another stream is still doing with it."""
    return _HERE if stream is None else torch.cuda.stream(stream)


def _ptr(t):
    return None if t is None else t.data_ptr()


def _size(t):
    return t.numel() * t.element_size()


# ----------------------------------------------------------------- API
@_plan
def _append_plan(k, v, kc, vc, tables, slots, rows, weights, positions, token_positions, group_size, bits):
    dims = _cache_dims(kc, vc, group_size, bits)
    heads, D = dims[4], dims[6]
    _dev(k, _BF16, "k", 3)
    _dev(v, _BF16, "v", 3)
    T = k[0][0]
    if k[0] != v[0] or tuple(k[0][1:]) != (heads, D):
        raise ValueError(f"k and v must be [T, {heads}, {D}], got {tuple(k[0])} and {tuple(v[0])}")
    B, cols = _dev(tables, _I32, "block_tables", 2)
    _whole(slots, _I32, "slots", (T,))
    if rows is not None:
        _whole(rows, _I32, "rows", (T,))
    elif T > B:
        raise ValueError(f"{T} tokens for {B} sequences: give rows")
    if token_positions is not None:
        _whole(token_positions, _I32, "token_positions", (T,))
    meta = (0, 0, 0)
    for t, dtype, name in ((weights, _F32, "weights"), (positions, _I32, "positions")):
        if t is None:
            continue
        _dev(t, dtype, name, 3)
        if tuple(t[0][:2]) != (B, heads):
            raise ValueError(f"{name} must be [{B}, {heads}, S], got {tuple(t[0])}")
        mine = _slots(t)
        if meta[2] and meta != mine:
            raise ValueError("weights and positions must have one shape and one layout")
        meta = mine
    _one_device(k, v, _first(kc), tables, slots, rows, weights, positions, token_positions)
    return dims, T, (tables[1][0] if B > 1 else cols, cols, B), meta


def qmv_kv_append(k, v, k_cache, v_cache, block_tables, slots, rows=None, weights=None, positions=None,
                  token_positions=None, group_size: int = 64, bits: int = 4, stream=None):
    """Write new tokens' keys and values, bf16 [T, heads, head_dim], into the
    cache, quantized on the way if it holds codes.  Token t goes to slot
    ``slots[t]`` of sequence ``rows[t]`` (sequence t without ``rows``); a negative
    slot is skipped.  ``weights`` and ``positions`` [B, heads, S], if given, get 0
    and ``token_positions[t]`` (or the slot) there: what ``qmv_kv_evict`` goes by."""
    dims, T, table, meta = _append_plan(
        _spec(k, "k"), _spec(v, "v"), _pool_spec(k_cache, "k_cache"), _pool_spec(v_cache, "v_cache"),
        _spec(block_tables, "block_tables"), _spec(slots, "slots"), _spec(rows, "rows"), _spec(weights, "weights"),
        _spec(positions, "positions"), _spec(token_positions, "token_positions"), group_size, bits)
    _call("qmv_kv_append", k.data_ptr(), k.stride(0), k.stride(1), v.data_ptr(), v.stride(0), v.stride(1),
          _cache(k_cache, v_cache, dims), block_tables.data_ptr(), *table, _ptr(rows), slots.data_ptr(), T, _ptr(weights),
          _ptr(positions), _ptr(token_positions), *meta, _stream(stream, k.device))


def qmv_kv_attend_workspace_bytes(k_cache, v_cache, block_tables, query_heads: int, weights: bool = False,
                                  max_length=None, group_size: int = 64, bits: int = 4) -> int:
    """Bytes of workspace that a ``qmv_kv_attend`` call of these sizes needs."""
    dims = _cache_dims(_pool_spec(k_cache, "k_cache"), _pool_spec(v_cache, "v_cache"), group_size, bits)
    return _attend_bytes(dims, block_tables.shape[0], block_tables.shape[1], query_heads // dims[4], int(weights),
                         int(max_length or 0))


@_plan
def _attend_plan(q, kc, vc, tables, lengths, mask, weights, weights_out, y, out_dtype, workspace, group_size, bits,
                 max_length):
    dims = _cache_dims(kc, vc, group_size, bits)
    heads = dims[4]
    B, Hq, D = _dev(q, _BF16, "q", 3)
    if D != dims[6] or Hq % heads or Hq == 0:
        raise ValueError(f"q must be [B, a multiple of {heads}, {dims[6]}], got {tuple(q[0])}")
    if _dev(tables, _I32, "block_tables", 2)[0] != B:
        raise ValueError(f"block_tables must have {B} rows, got {tables[0][0]}")
    cols = tables[0][1]
    _whole(lengths, _I32, "lengths", (B,))
    m = (0, 0, 0)
    if mask is not None:
        shape = tuple(_dev(mask, _F32, "mask"))
        if not 1 <= len(shape) <= 3:
            raise ValueError("mask must have 1 to 3 axes")
        shape, stride = (1,) * (3 - len(shape)) + shape, (0,) * (3 - len(shape)) + tuple(mask[1])
        if shape[0] not in (1, B) or shape[1] not in (1, Hq):
            raise ValueError(f"mask of shape {tuple(mask[0])} does not fit [{B}, {Hq}, slots]")
        m = (stride[0] if shape[0] > 1 else 0, stride[1] if shape[1] > 1 else 0, shape[2])
    w = (0, 0, 0)
    if weights is None:
        if weights_out is not None:
            raise ValueError("weights_out goes with weights")
    else:
        shape = _dev(weights, _F32, "weights", 3)
        if tuple(shape[:2]) != (B, heads):
            raise ValueError(f"weights must be [{B}, {heads}, S], got {tuple(shape)}")
        if weights_out is not None:
            _dev(weights_out, _F32, "weights_out", 3)
            if weights_out[0] != shape or _slots(weights_out) != _slots(weights):
                raise ValueError("weights and weights_out must have one shape and one layout")
        w = _slots(weights)
    code, dtype = _out_code(out_dtype)
    if y is not None:
        _whole(y, dtype, "y", (B, Hq, D))
    _workspace_ok(workspace)
    _one_device(q, _first(kc), tables, lengths, mask, weights, weights_out, y, workspace)
    group = Hq // heads
    need = _attend_bytes(dims, B, cols, group, int(weights is not None), max_length)
    return dims, (tables[1][0] if B > 1 else cols, cols), B, group, m, w, code, dtype, need


def qmv_kv_attend(q, k_cache, v_cache, block_tables, lengths, scale=None, mask=None, weights=None, weights_out=None,
                  group_size: int = 64, bits: int = 4, max_length=None, return_lse: bool = False, out_dtype=None,
                  y=None, workspace=None, stream=None):
    """Attention of one new token per sequence over its first ``lengths[b]`` slots.

    q: bf16 [B, query_heads, head_dim]; query heads are grouped over the
    cache's heads.  ``scale`` defaults to head_dim ** -0.5.  ``mask``: fp32,
    added to the scores, broadcastable to [B, query_heads, slots].  ``weights``:
    fp32 [B, heads, S], the attention each slot has had so far; the sum with
    this call's goes to ``weights_out`` (to ``weights`` itself without it).
    ``max_length``: the longest length, if known (a table wider than its
    sequences runs faster with it).  A query head with no slot gives y = 0 and
    lse = -inf.  Returns y, or (y, lse) with ``return_lse``."""
    most = int(max_length or 0)
    dims, table, B, group, m, w, code, dtype, need = _attend_plan(
        _spec(q, "q"), _pool_spec(k_cache, "k_cache"), _pool_spec(v_cache, "v_cache"),
        _spec(block_tables, "block_tables"), _spec(lengths, "lengths"), _spec(mask, "mask"), _spec(weights, "weights"),
        _spec(weights_out, "weights_out"), _spec(y, "y"), out_dtype, _spec(workspace, "workspace"), group_size, bits, most)
    device = q.device
    with _owner(stream):
        if y is None:
            y = q.new_empty(q.shape, dtype=dtype)
        lse = q.new_empty(q.shape[:2], dtype=_F32) if return_lse else None
        if workspace is None and need:
            workspace = q.new_empty(need, dtype=_U8)
    if weights_out is None:
        weights_out = weights
    _call("qmv_kv_attend", q.data_ptr(), q.stride(0), q.stride(1), _cache(k_cache, v_cache, dims),
          block_tables.data_ptr(), *table, lengths.data_ptr(), B, group,
          dims[6] ** -0.5 if scale is None else float(scale), _ptr(mask), *m, _ptr(weights), _ptr(weights_out), *w,
          y.data_ptr(), _ptr(lse), most, code, _ptr(workspace), 0 if workspace is None else _size(workspace),
          _stream(stream, device))
    return (y, lse) if return_lse else y


def qmv_kv_evict_workspace_bytes(B: int, heads: int, S: int, budget: int) -> int:
    """Bytes of workspace that a ``qmv_kv_evict`` call of these sizes needs."""
    return _bytes("qmv_kv_evict_workspace_bytes", B, heads, S, budget)


@_plan
def _evict_plan(kc, vc, tables, lengths, weights, positions, nxt, out, workspace, group_size, bits, budget):
    dims = _cache_dims(kc, vc, group_size, bits)
    heads = dims[4]
    B, cols = _dev(tables, _I32, "block_tables", 2)
    shape = _dev(weights, _F32, "weights", 3)
    _dev(positions, _I32, "positions", 3)
    S = shape[2]
    if tuple(shape[:2]) != (B, heads) or positions[0] != shape or S == 0:
        raise ValueError(f"weights and positions must be [{B}, {heads}, S], got {tuple(shape)} and {tuple(positions[0])}")
    if _slots(weights) != _slots(positions):
        raise ValueError("weights and positions must have one layout")
    _whole(lengths, _I32, "lengths", (B,))
    _whole(nxt, _I32, "next_positions", (B,))
    if out is not None:
        _whole(out[0], _I32, "out lengths", (B,))
        _whole(out[1], _F32, "out weights", shape)
        _whole(out[2], _I32, "out positions", shape)
        _one_device(tables, *out)
    _workspace_ok(workspace)
    _one_device(tables, _first(kc), lengths, weights, positions, nxt, workspace)
    return (dims, (tables[1][0] if B > 1 else cols, cols), B, _slots(weights),
            qmv_kv_evict_workspace_bytes(B, heads, S, budget))


def qmv_kv_evict(k_cache, v_cache, block_tables, lengths, weights, positions, next_positions, budget: int,
                 recent: int = 0, group_size: int = 64, bits: int = 4, out=None, workspace=None, stream=None):
    """Bring every sequence and head down to ``budget`` entries: the ``recent``
    newest by ``positions`` (those >= next_positions[b] - recent), then the
    heaviest ``weights``, ties to the lowest slot.  Keys and values move in
    place, survivors past the budget into the free slots below it.  weights,
    positions: fp32 and int32 [B, heads, S].  Returns (lengths, weights,
    positions) as they then are, in new tensors or the three of ``out``."""
    dims, table, B, meta, need = _evict_plan(
        _pool_spec(k_cache, "k_cache"), _pool_spec(v_cache, "v_cache"), _spec(block_tables, "block_tables"),
        _spec(lengths, "lengths"), _spec(weights, "weights"), _spec(positions, "positions"),
        _spec(next_positions, "next_positions"),
        None if out is None else tuple(_spec(t, "out") for t in out), _spec(workspace, "workspace"), group_size, bits,
        budget)
    device, shape = weights.device, weights.shape
    with _owner(stream):
        if out is None:
            out = lengths.new_empty(B), weights.new_empty(shape), positions.new_empty(shape)
        if workspace is None:
            workspace = weights.new_empty(need, dtype=_U8)
    _call("qmv_kv_evict", _cache(k_cache, v_cache, dims), block_tables.data_ptr(), *table, lengths.data_ptr(), B,
          weights.data_ptr(), positions.data_ptr(), *meta, next_positions.data_ptr(), budget, recent, out[0].data_ptr(),
          out[1].data_ptr(), out[2].data_ptr(), workspace.data_ptr(), _size(workspace), _stream(stream, device))
    return out


def qmv_beam_select_workspace_bytes(B: int, W: int, V: int, num: int) -> int:
    """Bytes of workspace that a ``qmv_beam_select`` call of these sizes needs."""
    return _bytes("qmv_beam_select_workspace_bytes", B, W, V, num)


@_plan
def _select_plan(logits, scores, num, out, workspace):
    if logits is None or logits[2] not in (_BF16, _F32):
        raise ValueError("logits must be a bf16 or fp32 device tensor")
    B, W, V = _dev(logits, logits[2], "logits", 3)
    stride = logits[1]
    ld = stride[1] if W > 1 else (stride[0] if B > 1 else V)
    if W > 1 and B > 1 and stride[0] != W * ld:
        raise ValueError("logits: beams must follow each other at one stride")
    _whole(scores, _F32, "scores", (B, W))
    if out is not None:
        for t, dtype, name in zip(out, (_F32, _I32, _I32), ("scores", "beams", "tokens")):
            _whole(t, dtype, f"out {name}", (B, num))
        _one_device(logits, *out)
    _workspace_ok(workspace)
    _one_device(logits, scores, workspace)
    return (QMV_OUT_F32 if logits[2] == _F32 else QMV_OUT_BF16, ld), (B, W, V), qmv_beam_select_workspace_bytes(B, W, V, num)


def qmv_beam_select(logits, scores, num: int, out=None, workspace=None, stream=None):
    """The best ``num`` (at most 32) of W beams x V tokens by
    ``scores[b, w] + log_softmax(logits[b, w])[v]``, ties to the lowest
    w * V + v.  logits: bf16 or fp32 [B, W, V]; scores: fp32 [B, W].  Returns
    (scores fp32, beams int32, tokens int32), each [B, num], best first."""
    form, sizes, need = _select_plan(
        _spec(logits, "logits"), _spec(scores, "scores"), num,
        None if out is None else tuple(_spec(t, "out") for t in out), _spec(workspace, "workspace"))
    device = logits.device
    with _owner(stream):
        if out is None:
            shape = (sizes[0], num)
            out = scores.new_empty(shape), scores.new_empty(shape, dtype=_I32), scores.new_empty(shape, dtype=_I32)
        if workspace is None:
            workspace = scores.new_empty(need, dtype=_U8)
    _call("qmv_beam_select", logits.data_ptr(), *form, scores.data_ptr(), *sizes, num, out[0].data_ptr(),
          out[1].data_ptr(), out[2].data_ptr(), workspace.data_ptr(), _size(workspace), _stream(stream, device))
    return out


@_plan
def _reorder_plan(kc, vc, tables, lengths, parents, spare, out, group_size, bits):
    dims = _cache_dims(kc, vc, group_size, bits)
    B, W, cols = _dev(tables, _I32, "block_tables", 3)
    _whole(tables, _I32, "block_tables", (B, W, cols))
    _whole(lengths, _I32, "lengths", (B, W))
    M = _dev(parents, _I32, "parents", 2)[1]
    if parents[0][0] != B or M == 0:
        raise ValueError(f"parents must be [{B}, M], got {tuple(parents[0])}")
    _whole(spare, _I32, "spare_pages", (B, M))
    if out is not None:
        _whole(out[0], _I32, "out block_tables", (B, M, cols))
        _whole(out[1], _I32, "out lengths", (B, M))
        _one_device(tables, *out)
    _one_device(tables, _first(kc), lengths, parents, spare)
    return dims, (B, W, cols), (parents[1][0] if B > 1 else M, M)


def qmv_beam_reorder(k_cache, v_cache, block_tables, lengths, parents, spare_pages, group_size: int = 64,
                     bits: int = 4, out=None, stream=None):
    """New beam i of item b continues beam ``parents[b, i]``: it shares that
    beam's full pages and gets a copy of its last, partly filled one in page
    ``spare_pages[b, i]``, which becomes its last page (empty if the parent's was
    full).  block_tables: int32 [B, W, columns]; lengths: [B, W]; parents,
    spare_pages: [B, M].  Returns (block_tables [B, M, columns], lengths
    [B, M]); entries past the last page are -1."""
    dims, sizes, par = _reorder_plan(
        _pool_spec(k_cache, "k_cache"), _pool_spec(v_cache, "v_cache"), _spec(block_tables, "block_tables"),
        _spec(lengths, "lengths"), _spec(parents, "parents"), _spec(spare_pages, "spare_pages"),
        None if out is None else tuple(_spec(t, "out") for t in out), group_size, bits)
    device = lengths.device
    with _owner(stream):
        if out is None:
            out = lengths.new_empty((sizes[0], par[1], sizes[2])), lengths.new_empty((sizes[0], par[1]))
    _call("qmv_beam_reorder", _cache(k_cache, v_cache, dims), block_tables.data_ptr(), lengths.data_ptr(), *sizes,
          parents.data_ptr(), *par, spare_pages.data_ptr(), out[0].data_ptr(), out[1].data_ptr(), _stream(stream, device))
    return out
