"""Binding of the latent-row operators (include/sfa_grad.h): the norm and
position rotation of the attention's input rows with their gradients, the
append to a paged cache of 16 or 4 bits, the attention of new tokens over it,
and the block tables and slot maps of a step.  Argument checks and marshalling
only, like the rest of the binding.
"""
from __future__ import annotations

import ctypes
import functools
import struct
from typing import Optional

import torch

from . import DTYPES, LAYOUTS, _check, _stream, _workspace, lib

EXPORTS = ("sfa_norm_rope", "sfa_norm_rope_grad_workspace_size", "sfa_norm_rope_grad", "sfa_cache_append",
           "sfa_paged_workspace_size", "sfa_paged_fwd", "sfa_norm_rope_axes", "sfa_norm_rope_axes_grad",
           "sfa_cache4_append", "sfa_paged4_workspace_size", "sfa_paged4_fwd", "sfa_cache4_unpack",
           "sfa_cache_append_slots", "sfa_page_plan")

CODES4 = 288        # bytes of a 4-bit row before its rotated part: 256 of codes, 32 of scales


class RowsParams(ctypes.Structure):
    _fields_ = [("dtype", ctypes.c_int32), ("interleaved", ctypes.c_int32), ("T1", ctypes.c_int64),
                ("N1", ctypes.c_int64), ("table_len", ctypes.c_int64), ("eps", ctypes.c_double)]


class PagedParams(ctypes.Structure):
    _fields_ = [("layout", ctypes.c_int32), ("dtype", ctypes.c_int32),
                ("B", ctypes.c_int64), ("S1", ctypes.c_int64), ("T1", ctypes.c_int64),
                ("N1", ctypes.c_int64), ("D", ctypes.c_int64), ("Dr", ctypes.c_int64),
                ("num_pages", ctypes.c_int64), ("page_size", ctypes.c_int64), ("max_pages", ctypes.c_int64),
                ("scale", ctypes.c_double), ("sparse_mode", ctypes.c_int64),
                ("interleaved", ctypes.c_int32), ("wait_limit_us", ctypes.c_int32)]


class CacheParams(ctypes.Structure):
    _fields_ = [("dtype", ctypes.c_int32), ("bits", ctypes.c_int32), ("num_pages", ctypes.c_int64),
                ("page_size", ctypes.c_int64), ("Dr", ctypes.c_int64), ("scale", ctypes.c_double)]


class PlanParams(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int64), ("max_pages", ctypes.c_int64), ("num_pages", ctypes.c_int64),
                ("page_size", ctypes.c_int64), ("tokens", ctypes.c_int64)]


# The calls pass their parameters packed: a Structure costs more to fill than
# the whole of a small call's checks.
_pack_rows = struct.Struct("@iiqqqd").pack
_pack_paged = struct.Struct("@iiqqqqqqqqqdqii").pack
_pack_cache = struct.Struct("@iiqqqd").pack
_pack_plan = struct.Struct("@qqqqq").pack
assert struct.calcsize("@iiqqqd") == ctypes.sizeof(RowsParams) == ctypes.sizeof(CacheParams)
assert struct.calcsize("@qqqqq") == ctypes.sizeof(PlanParams)
assert struct.calcsize("@iiqqqqqqqqqdqii") == ctypes.sizeof(PagedParams)

_ready = None


def _lib():
    global _ready
    if _ready is None:
        L = lib()
        vp, sz, d, i64 = ctypes.c_void_p, ctypes.c_size_t, ctypes.c_double, ctypes.c_int64
        R = P = vp
        L.sfa_norm_rope.argtypes = [R] + [vp] * 15
        L.sfa_norm_rope_grad_workspace_size.argtypes = [R, ctypes.POINTER(sz)]
        L.sfa_norm_rope_grad.argtypes = [R] + [vp] * 18 + [vp, sz, vp]
        L.sfa_cache_append.argtypes = [P] + [vp] * 7 + [d, vp, i64] + [vp] * 4
        L.sfa_paged_workspace_size.argtypes = [P, ctypes.POINTER(sz)]
        L.sfa_paged_fwd.argtypes = [P] + [vp] * 10 + [sz, vp]
        i32 = ctypes.c_int32
        L.sfa_norm_rope_axes.argtypes = [R, i32] + [vp] * 16
        L.sfa_norm_rope_axes_grad.argtypes = [R, i32] + [vp] * 19 + [vp, sz, vp]
        L.sfa_cache4_append.argtypes = [P, d] + [vp] * 7 + [d, vp, i64] + [vp] * 4
        L.sfa_paged4_workspace_size.argtypes = [P, ctypes.POINTER(sz)]
        L.sfa_paged4_fwd.argtypes = [P, d] + [vp] * 10 + [sz, vp]
        L.sfa_cache4_unpack.argtypes = [vp] * 4
        L.sfa_cache_append_slots.argtypes = [vp, R, vp, vp, i32] + [vp] * 10
        L.sfa_page_plan.argtypes = [vp] * 13
        for name in EXPORTS:
            getattr(L, name).restype = ctypes.c_int32
        _ready = L
    return _ready


# A call on few rows takes the GPU a few microseconds, so the checks below are
# written to cost little: one comparison a property, messages only on failure,
# devices as their indices (-1: the CPU), and empty_strided for what is not
# like an input (half of what torch.empty costs).
def _need(name: str, t: Optional[torch.Tensor], shape, dtype, index):
    """Checks a tensor and returns its address."""
    if t is None:
        raise ValueError(f"{name} is required")
    if t.dtype is dtype and t.shape == shape and t.get_device() == index and t.is_contiguous():
        return t.data_ptr()
    if t.dtype is not dtype:
        raise ValueError(f"{name}: dtype {t.dtype}, expected {dtype}")
    if t.shape != shape:
        raise ValueError(f"{name}: shape {tuple(t.shape)}, expected {tuple(shape)}")
    if t.get_device() != index:
        raise ValueError(f"{name} is on {t.device}, expected " + (f"cuda:{index}" if index >= 0 else "cpu"))
    raise ValueError(f"{name}: tensors must be contiguous")


def _floats(shape, like):
    strides, n = [], 1
    for k in reversed(shape):
        strides.append(n)
        n *= k
    return torch.empty_strided(shape, strides[::-1], dtype=torch.float32, device=like.device)


def _on_stream(fn):
    """Makes `stream` the current one for the call, so that what the call
    allocates itself (outputs, workspace) belongs to that stream."""
    @functools.wraps(fn)
    def call(*args, stream=None, **kw):
        if stream is None:
            return fn(*args, **kw)
        with torch.cuda.stream(stream):
            return fn(*args, stream=stream, **kw)
    return call


def _call(index, stream, fn, what, *args):
    """fn(*args, stream handle) with the tensors' device current."""
    if index < 0:
        raise ValueError("tensors must live on a CUDA device")
    if stream is not None and stream.device.index != index:
        raise ValueError(f"stream is on {stream.device}, the call runs on cuda:{index}")
    if index == torch._C._cuda_getDevice():
        rc = fn(*args, torch._C._cuda_getCurrentRawStream(index))
    else:
        with torch.cuda.device(index):
            rc = fn(*args, _stream(None))
    if rc:
        _check(rc, what)


# ------------------------------------------------------------------ norm and rotation
def _axes(axes, positions, tokens):
    """Number of axes, and the axis of each pair as 32 bytes."""
    at = bytes(tuple(axes))
    if positions is None or positions.dim() < 1 or positions.numel() != positions.shape[0] * tokens:
        raise ValueError(f"positions: expected (axes, ...) of {tokens} tokens")
    n = positions.shape[0]
    if not 1 <= n <= 4:
        raise ValueError(f"positions: {n} axes, expected 1 to 4")
    if len(at) != 32 or max(at) >= n:
        raise ValueError(f"axes: expected 32 numbers below {n}, the axis of each rotated pair")
    return n, at


def _rows(q, q_rope, k, k_rope, positions, cos_sin, eps, interleaved, axes=None):
    """Parameters, leading shape, heads and addresses of the row tensors that
    are there (queries (..., N1, 512 / 64), keys (..., 1, 512 / 64))."""
    first = k if k is not None else q if q is not None else k_rope if k_rope is not None else q_rope
    if first is None:
        raise ValueError("at least one of q, q_rope, k, k_rope is required")
    dt, dev = first.dtype, first.get_device()
    if dt not in DTYPES:
        raise ValueError("rows must be bfloat16 or float16")
    if first.dim() < 2:
        raise ValueError("rows need a head dimension: (..., heads, 512) or (..., heads, 64)")
    lead = first.shape[:-2]
    heads = q.shape[-2] if q is not None else q_rope.shape[-2] if q_rope is not None else 1
    at = (None if q is None else _need("q", q, lead + (heads, 512), dt, dev),
          None if q_rope is None else _need("q_rope", q_rope, lead + (heads, 64), dt, dev),
          None if k is None else _need("k", k, lead + (1, 512), dt, dev),
          None if k_rope is None else _need("k_rope", k_rope, lead + (1, 64), dt, dev))
    tokens = lead.numel()
    if (positions is None or cos_sin is None) and (q_rope is not None or k_rope is not None):
        raise ValueError("positions and cos_sin are required with q_rope or k_rope")
    pos = cs = None
    table_len = 0
    if positions is not None:
        if axes is None and positions.numel() != tokens:
            raise ValueError(f"positions: {positions.numel()} elements, expected {tokens}")
        pos = _need("positions", positions, positions.shape, torch.int32, dev)
        if cos_sin is None:
            raise ValueError("cos_sin is required with positions")
    if cos_sin is not None:
        table_len = cos_sin.shape[0]
        cs = _need("cos_sin", cos_sin, (table_len, 64), torch.float32, dev)
    return (DTYPES[dt], 1 if interleaved else 0, tokens, heads, table_len, eps), lead, heads, dt, dev, pos, cs, at


@_on_stream
def norm_rope(positions, cos_sin, *, k=None, k_weight=None, k_rope=None, q=None, q_weight=None, q_rope=None, eps=1e-6,
              interleaved=True, outputs=None, axes=None, stream=None):
    """sfa_norm_rope on torch CUDA tensors: normalises k (..., 1, 512) and q
    (..., N1, 512) by their weights (512,), rotates k_rope (..., 1, 64) and
    q_rope (..., N1, 64) by cos_sin[positions] (fp32 (P, 64): 32 cosines, 32
    sines).  Each of the four rows may be left out.  Returns (q, q_rope, k,
    k_rope, q_rstd, k_rstd), None where its input is; `outputs`: such a tuple
    to write into, where an output may be its own input.  `axes`: 32 numbers,
    the axis of each rotated pair; positions then are (axes, ...), up to four
    of them (sfa_norm_rope_axes)."""
    p, lead, heads, dt, dev, pos, cs, (qa, qra, ka, kra) = _rows(q, q_rope, k, k_rope, positions, cos_sin, eps,
                                                                 interleaved, axes)
    kw = None if k is None else _need("k_weight", k_weight, (512,), dt, dev)
    qw = None if q is None else _need("q_weight", q_weight, (512,), dt, dev)
    if outputs is None:
        outputs = (None if q is None else torch.empty_like(q), None if q_rope is None else torch.empty_like(q_rope),
                   None if k is None else torch.empty_like(k), None if k_rope is None else torch.empty_like(k_rope),
                   None if q is None else _floats(lead + (heads,), q),
                   None if k is None else _floats(lead + (1,), k))
        o = [None if t is None else t.data_ptr() for t in outputs]
    else:
        o = [None if x is None else _need(f"outputs: {name}", t, x.shape, dt, dev)
             for name, t, x in zip(("q", "q_rope", "k", "k_rope"), outputs, (q, q_rope, k, k_rope))]
        o += [None if x is None or t is None else _need(f"outputs: {name}", t, lead + (h,), torch.float32, dev)
              for name, t, x, h in (("q_rstd", outputs[4], q, heads), ("k_rstd", outputs[5], k, 1))]
    if axes is None:
        _call(dev, stream, _lib().sfa_norm_rope, "sfa_norm_rope", _pack_rows(*p), pos, cs, qa, qw, qra, ka, kw, kra, *o)
    else:
        _call(dev, stream, _lib().sfa_norm_rope_axes, "sfa_norm_rope_axes", _pack_rows(*p),
              *_axes(axes, positions, p[2]), pos, cs, qa, qw, qra, ka, kw, kra, *o)
    return outputs


@_on_stream
def norm_rope_grad(positions, cos_sin, *, k=None, k_weight=None, k_rstd=None, dk=None, dk_rope=None, q=None,
                   q_weight=None, q_rstd=None, dq=None, dq_rope=None, interleaved=True, workspace=None, axes=None,
                   stream=None):
    """sfa_norm_rope_grad: gradients of norm_rope's inputs from those of its
    outputs (dq, dq_rope, dk, dk_rope, for instance sfa_grad's; where the row
    is key and value, dk is the sum of its dK and dV).  k, k_weight and k_rstd
    (q, ...) are norm_rope's inputs and its saved rstd, positions and axes as
    there.  Returns (dq, dq_rope, dk, dk_rope, dq_weight, dk_weight); the
    weights' gradients are fp32, summed in a fixed order."""
    p, lead, heads, dt, dev, pos, cs, (dqa, dqra, dka, dkra) = _rows(dq, dq_rope, dk, dk_rope, positions, cos_sin, 0.0,
                                                                     interleaved, axes)
    several = () if axes is None else _axes(axes, positions, p[2])
    saved = {}
    for name, d, x, w, r, h in (("k", dk, k, k_weight, k_rstd, 1), ("q", dq, q, q_weight, q_rstd, heads)):
        saved[name] = (None, None, None) if d is None else (
            _need(name, x, d.shape, dt, dev), _need(f"{name}_weight", w, (512,), dt, dev),
            _need(f"{name}_rstd", r, lead + (h,), torch.float32, dev))
    out = [None if d is None else torch.empty_like(d) for d in (dq, dq_rope, dk, dk_rope)]
    out += [None if d is None else _floats((512,), d) for d in (dq, dk)]
    if p[2] == 0:      # no token: the weights' gradients are empty sums
        for t in out[4:]:
            if t is not None:
                t.zero_()
        return tuple(out)
    ws, nbytes = None, 0
    if dq is not None or dk is not None:
        if workspace is None or workspace.get_device() != dev:
            workspace = _workspace(norm_rope_grad_workspace_size(RowsParams(*p)), (dk if dq is None else dq).device,
                                   workspace)
        ws, nbytes = _need("workspace", workspace, workspace.shape, workspace.dtype, dev), \
            workspace.numel() * workspace.element_size()
    o = [None if t is None else t.data_ptr() for t in out]
    fn, what = (_lib().sfa_norm_rope_axes_grad, "sfa_norm_rope_axes_grad") if several else \
        (_lib().sfa_norm_rope_grad, "sfa_norm_rope_grad")
    _call(dev, stream, fn, what, _pack_rows(*p), *several, pos, cs, *saved["q"], *saved["k"], dqa, dqra, dka, dkra, *o,
          ws, nbytes)
    return tuple(out)


def norm_rope_grad_workspace_size(p: RowsParams) -> int:
    n = ctypes.c_size_t(0)
    _check(_lib().sfa_norm_rope_grad_workspace_size(ctypes.byref(p), ctypes.byref(n)),
           "sfa_norm_rope_grad_workspace_size")
    return n.value


# ------------------------------------------------------------------ paged cache
def make_paged_params(cache, block_table, act_seq_kv, *, tokens, heads, layout="BSND", seq=None, act_seq_q=None,
                      scale=1.0, sparse_mode=3, interleaved=True, wait_limit_us=0, dtype=None) -> PagedParams:
    """Parameters of the paged calls, with checks of the cache and of the index
    tensors.  `tokens`: rows of q (B * S1 for BSND, with `seq` = S1); `dtype`:
    theirs, for a cache of 4 bits."""
    if cache.dtype is torch.uint8 and dtype is None:
        raise ValueError("dtype is required for a cache of 4 bits")
    return PagedParams(*_paged(cache, block_table, act_seq_kv, tokens, heads, layout, seq, act_seq_q, scale,
                               sparse_mode, interleaved, wait_limit_us, dtype)[0])


def _cache(cache, dtype, cache_scale):
    """dtype of the rows, width of their rotated part, the scale of a cache of
    4 bits (None: 16 bits), and the cache's shape."""
    held, shape = cache.dtype, cache.shape
    if held in DTYPES:
        if len(shape) != 3 or shape[2] not in (512, 576):
            raise ValueError("cache: expected (num_pages, page_size, 576) or (num_pages, page_size, 512)")
        if cache_scale is not None:
            raise ValueError("cache_scale given for a cache of 16 bits")
        return held, shape[2] - 512, None, shape
    if held is not torch.uint8:
        raise ValueError("cache must be bfloat16 or float16, or uint8 (rows of 4 bits)")
    if len(shape) != 3 or shape[2] not in (CODES4, CODES4 + 128):
        raise ValueError("cache of 4 bits: expected (num_pages, page_size, 416) or (num_pages, page_size, 288)")
    if dtype not in DTYPES:
        raise ValueError("rows must be bfloat16 or float16")
    return dtype, (shape[2] - CODES4) // 2, 1.0 if cache_scale is None else cache_scale, shape


def _paged(cache, block_table, act_seq_kv, tokens, heads, layout, seq, act_seq_q, scale, sparse_mode, interleaved,
           wait_limit_us, dtype=None, cache_scale=None):
    """The fields of PagedParams, the addresses of cache, block_table,
    act_seq_q and act_seq_kv, of a cache of 4 bits its scale, and the rows'
    dtype and device."""
    dt, dr, unit, shape = _cache(cache, dtype, cache_scale)
    if block_table.dim() != 2:
        raise ValueError("block_table: expected (B, max_pages)")
    dev = cache.get_device()
    pages, page, _ = shape
    b, per = entries = block_table.shape
    at = (_need("cache", cache, shape, dt if unit is None else torch.uint8, dev),
          _need("block_table", block_table, entries, torch.int32, dev))
    kva = _need("act_seq_kv", act_seq_kv, (b,), torch.int32, dev)
    lay = LAYOUTS[layout.upper()]
    qla = None
    if act_seq_q is not None or lay == 1:
        qla = _need("act_seq_q", act_seq_q, (b,), torch.int32, dev)
    if lay == 0 and tokens != b * seq:
        raise ValueError(f"BSND rows of {tokens} tokens do not match {b} sequences of {seq}")
    return (lay, DTYPES[dt], b, 0 if lay else seq, tokens if lay else 0, heads, 512, dr, pages, page, per, scale,
            sparse_mode, 1 if interleaved else 0, wait_limit_us), at + (qla, kva), unit, dt, dev


def _leading(name, t, layout):
    """Leading shape of rows in a layout, tokens and S1."""
    n = 2 if layout.upper() == "BSND" else 1
    if t.dim() != n + 2:
        raise ValueError(f"{name}: expected {'(B, S1' if n == 2 else '(T1'}, heads, width)")
    lead = t.shape[:n]
    tokens = lead[0] * (lead[1] if n == 2 else 1)
    return lead, tokens, lead[1] if n == 2 else None


@_on_stream
def cache_append(cache, block_table, act_seq_kv, k, k_rope=None, cos_sin=None, *, k_weight=None, eps=1e-6,
                 interleaved=True, q_rope=None, q_rope_out=None, layout="BSND", act_seq_q=None, error=None,
                 cache_scale=None, stream=None):
    """sfa_cache_append: writes the new tokens' rows [norm(k) || rotated
    k_rope] into `cache`, (num_pages, page_size, 576 or 512) or, of 4 bits in
    units of cache_scale (a power of two; 1 unless given), uint8 (num_pages,
    page_size, 416 or 288) (sfa_cache4_append); k is (B, S1, 1,
    512) or (T1, 1, 512).  act_seq_kv counts the new tokens too, and their
    positions are the last of their sequences.  With q_rope (..., N1, 64) the
    same launch rotates it into q_rope_out (allocated unless given; q_rope
    itself is allowed).  `error`: optional int32 (1,) that receives a
    SFA_DEVERR_* code.  Returns (cache, q_rope_out)."""
    lead, tokens, seq = _leading("k", k, layout)
    heads = 1 if q_rope is None else q_rope.shape[-2]
    p, (ca, bta, aq, akv), unit, dt, dev = _paged(cache, block_table, act_seq_kv, tokens, heads, layout, seq, act_seq_q,
                                                  1.0, 3, interleaved, 0, k.dtype, cache_scale)
    (ka, kra, kw, cs, qra, qroa), table_len, err, q_rope_out = _new_rows(
        dt, dev, p[7], lead, heads, k, k_rope, k_weight, cos_sin, q_rope, q_rope_out, error)
    args = (ca, bta, aq, akv, ka, kra, kw, eps, cs, table_len, qra, qroa, err)
    if unit is None:
        _call(dev, stream, _lib().sfa_cache_append, "sfa_cache_append", _pack_paged(*p), *args)
    else:
        _call(dev, stream, _lib().sfa_cache4_append, "sfa_cache4_append", _pack_paged(*p), unit, *args)
    return cache, q_rope_out


def _new_rows(dt, dev, dr, lead, heads, k, k_rope, k_weight, cos_sin, q_rope, q_rope_out, error):
    """Addresses of an append's rows, its table's length and error word, and
    q_rope_out."""
    ka = _need("k", k, lead + (1, 512), dt, dev)
    kw = None if k_weight is None else _need("k_weight", k_weight, (512,), dt, dev)
    kra = cs = qra = qroa = None
    table_len = 0
    if dr:
        kra = _need("k_rope", k_rope, lead + (1, 64), dt, dev)
        if cos_sin is None:
            raise ValueError("cos_sin is required")
        table_len = cos_sin.shape[0]
        cs = _need("cos_sin", cos_sin, (table_len, 64), torch.float32, dev)
        if q_rope is not None:
            qra = _need("q_rope", q_rope, lead + (heads, 64), dt, dev)
            if q_rope_out is None:
                q_rope_out = torch.empty_like(q_rope)
            qroa = _need("q_rope_out", q_rope_out, lead + (heads, 64), dt, dev)
    elif k_rope is not None or q_rope is not None:
        raise ValueError("rope rows given for a cache without them")
    err = None if error is None else _need("error", error, (1,), torch.int32, dev)
    return (ka, kra, kw, cs, qra, qroa), table_len, err, q_rope_out


@_on_stream
def cache_append_slots(cache, slots, positions, k, k_rope=None, cos_sin=None, *, k_weight=None, eps=1e-6,
                       interleaved=True, q_rope=None, q_rope_out=None, axes=None, error=None, cache_scale=None,
                       stream=None):
    """sfa_cache_append_slots: as cache_append, with the rows' places in a slot
    map (tokens,) int32 (page_plan's, for instance; negative: padding, left
    out) and their positions given, (tokens,) or, with `axes` (32 numbers, the
    axis of each rotated pair), (axes, tokens).  k is (tokens, 1, 512).
    Positions are not needed for a cache without rotated rows.  Returns (cache,
    q_rope_out)."""
    dt, dr, unit, shape = _cache(cache, k.dtype, cache_scale)
    dev = cache.get_device()
    if k.dim() != 3:
        raise ValueError("k: expected (tokens, 1, 512)")
    lead, tokens = k.shape[:1], k.shape[0]
    heads = 1 if q_rope is None else q_rope.shape[-2]
    ca = _need("cache", cache, shape, cache.dtype, dev)
    sa = _need("slots", slots, (tokens,), torch.int32, dev)
    (ka, kra, kw, cs, qra, qroa), table_len, err, q_rope_out = _new_rows(
        dt, dev, dr, lead, heads, k, k_rope, k_weight, cos_sin, q_rope, q_rope_out, error)
    n, at, pos = 1, None, None
    if dr:
        if positions is None:
            raise ValueError("positions is required")
        if axes is not None:
            n, at = _axes(axes, positions, tokens)
        pos = _need("positions", positions, (tokens,) if axes is None else (n, tokens), torch.int32, dev)
    elif axes is not None:
        raise ValueError("axes given for a cache without rope rows")
    pages, page, _ = shape
    _call(dev, stream, _lib().sfa_cache_append_slots, "sfa_cache_append_slots",
          _pack_cache(DTYPES[dt], 16 if unit is None else 4, pages, page, dr, 0.0 if unit is None else unit),
          _pack_rows(DTYPES[dt], 1 if interleaved else 0, tokens, heads, table_len, eps), ca, sa, n, at, pos, ka, kra,
          kw, cs, qra, qroa, err)
    return cache, q_rope_out


@_on_stream
def cache_unpack(cache, dtype, *, cache_scale=None, out=None, stream=None):
    """sfa_cache4_unpack: the values of a 4-bit cache, (num_pages, page_size,
    576 or 512) in dtype, which is the one its rows were appended in."""
    if cache.dtype is not torch.uint8:
        raise ValueError("cache must be uint8 (rows of 4 bits)")
    dt, dr, unit, held = _cache(cache, dtype, cache_scale)
    dev = cache.get_device()
    shape = held[:2] + (512 + dr,)
    if out is None:
        out = torch.empty(shape, dtype=dt, device=cache.device)
    _call(dev, stream, _lib().sfa_cache4_unpack, "sfa_cache4_unpack",
          _pack_cache(DTYPES[dt], 4, shape[0], shape[1], dr, unit),
          _need("cache", cache, held, torch.uint8, dev), _need("out", out, shape, dt, dev))
    return out


# ------------------------------------------------------------------ a step's tables
@_on_stream
def page_plan(block_table, act_seq_kv, new_tokens, free_pages, free_count, *, page_size, tokens, error=None,
              outputs=None, stream=None):
    """sfa_page_plan: gives the requests of a step the pages that their new
    tokens need and takes back those of ended ones (new_tokens negative), on
    the device.  block_table (B, max_pages) and free_pages (num_pages,), of
    which the first free_count (1,) are free, are changed in place; all int32.
    Returns (act_seq_q, act_seq_kv, free_count, slots, positions): the new
    tokens and lengths of the step, what is left, and the row of the cache and
    position of each new token, `tokens` of them (-1 behind the last).
    `outputs`: such a tuple to write into, none of them an input.  `error`:
    optional int32 (1,) that receives a SFA_DEVERR_* code; a step that does not
    fit changes nothing.  A request holds the pages of its act_seq_kv tokens: a
    length that is lowered between steps stays within its last page, or the
    caller returns the pages behind it; pages that requests share come back
    from each of them."""
    if block_table.dim() != 2 or free_pages.dim() != 1:
        raise ValueError("expected block_table (B, max_pages) and free_pages (num_pages,)")
    b, per = block_table.shape
    dev, i32 = block_table.get_device(), torch.int32
    at = (_need("block_table", block_table, block_table.shape, i32, dev),
          _need("act_seq_kv", act_seq_kv, (b,), i32, dev), _need("new_tokens", new_tokens, (b,), i32, dev),
          _need("free_pages", free_pages, free_pages.shape, i32, dev),
          _need("free_count", free_count, (1,), i32, dev))
    if outputs is None:
        if tokens < 0:
            raise ValueError("tokens must not be negative")
        # (new_empty, or the parts of one allocation, took 8 and 3 us longer)
        new, device = torch.empty_strided, block_table.device
        outputs = tuple(new((n,), (1,), dtype=i32, device=device) for n in (b, b, 1, tokens, tokens))
        o = [t.data_ptr() for t in outputs]
    else:
        o = [_need(f"outputs: {name}", t, shape, i32, dev) for name, t, shape in
             zip(("act_seq_q", "act_seq_kv", "free_count", "slots", "positions"), outputs,
                 ((b,), (b,), (1,), (tokens,), (tokens,)))]
    err = None if error is None else _need("error", error, (1,), i32, dev)
    _call(dev, stream, _lib().sfa_page_plan, "sfa_page_plan",
          _pack_plan(b, per, free_pages.shape[0], page_size, tokens), *at, *o, err)
    return outputs


# ------------------------------------------------------------------ attention over the cache
def paged4_workspace_size(p: PagedParams) -> int:
    n = ctypes.c_size_t(0)
    _check(_lib().sfa_paged4_workspace_size(ctypes.byref(p), ctypes.byref(n)), "sfa_paged4_workspace_size")
    return n.value


def paged_workspace_size(p: PagedParams) -> int:
    n = ctypes.c_size_t(0)
    _check(_lib().sfa_paged_workspace_size(ctypes.byref(p), ctypes.byref(n)), "sfa_paged_workspace_size")
    return n.value


@_on_stream
def paged_fwd(q, cache, block_table, act_seq_kv, scale, *, q_rope=None, layout="BSND", act_seq_q=None, sparse_mode=3,
              out=None, softmax_max=None, softmax_sum=None, workspace=None, stream=None, wait_limit_us=0,
              cache_scale=None):
    """sfa_paged_fwd: attention of the new tokens' q (B, S1, N1, 512) or (T1,
    N1, 512) over their sequences' rows in the paged cache; returns (out,
    softmax_max, softmax_sum), the statistics (B, 1, S1, N1) or (1, T1, N1) as
    fwd's.  Rows of no sequence (BSND past act_seq_q, TND past the last
    sequence) are left as they were.  A uint8 cache holds rows of 4 bits in
    units of cache_scale, as cache_append's (sfa_paged4_fwd).
    read_device_error reads a passed workspace's error word."""
    lead, tokens, seq = _leading("q", q, layout)
    heads = q.shape[-2]
    p, (ca, bta, aq, akv), unit, dt, dev = _paged(cache, block_table, act_seq_kv, tokens, heads, layout, seq, act_seq_q,
                                                  scale, sparse_mode, True, wait_limit_us, q.dtype, cache_scale)
    qa = _need("q", q, lead + (heads, 512), dt, dev)
    qra = None
    if p[7]:
        qra = _need("q_rope", q_rope, lead + (heads, 64), dt, dev)
    elif q_rope is not None:
        raise ValueError("q_rope given for a cache without rope rows")
    st_shape = (lead[0], 1, lead[1], heads) if seq is not None else (1, tokens, heads)
    if out is None:
        out = torch.empty_like(q)
    oa = _need("out", out, q.shape, dt, dev)
    if softmax_max is None:
        softmax_max = _floats(st_shape, q)
    if softmax_sum is None:
        softmax_sum = torch.empty_like(softmax_max)
    ma = _need("softmax_max", softmax_max, st_shape, torch.float32, dev)
    sa = _need("softmax_sum", softmax_sum, st_shape, torch.float32, dev)
    if workspace is None or workspace.get_device() != dev:
        size = paged_workspace_size if unit is None else paged4_workspace_size
        workspace = _workspace(size(PagedParams(*p)), cache.device, workspace)
    ws = _need("workspace", workspace, workspace.shape, workspace.dtype, dev)
    args = (qa, qra, ca, bta, aq, akv, oa, ma, sa, ws, workspace.numel() * workspace.element_size())
    if unit is None:
        _call(dev, stream, _lib().sfa_paged_fwd, "sfa_paged_fwd", _pack_paged(*p), *args)
    else:
        _call(dev, stream, _lib().sfa_paged4_fwd, "sfa_paged4_fwd", _pack_paged(*p), unit, *args)
    return out, softmax_max, softmax_sum
