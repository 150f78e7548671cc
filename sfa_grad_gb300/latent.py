"""Binding of the latent-row operators (include/sfa_grad.h): the norm and
position rotation of the attention's input rows with their gradients, the
append to a paged cache, and the attention of new tokens over it.  Argument
checks and marshalling only, like the rest of the binding.
"""
from __future__ import annotations

import ctypes
import functools
import struct
from typing import Optional

import torch

from . import DTYPES, LAYOUTS, _check, _stream, _workspace, lib

EXPORTS = ("sfa_norm_rope", "sfa_norm_rope_grad_workspace_size", "sfa_norm_rope_grad", "sfa_cache_append",
           "sfa_paged_workspace_size", "sfa_paged_fwd")


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


# The calls pass their parameters packed: a Structure costs more to fill than
# the whole of a small call's checks.
_pack_rows = struct.Struct("@iiqqqd").pack
_pack_paged = struct.Struct("@iiqqqqqqqqqdqii").pack
assert struct.calcsize("@iiqqqd") == ctypes.sizeof(RowsParams)
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
def _rows(q, q_rope, k, k_rope, positions, cos_sin, eps, interleaved):
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
        if positions.numel() != tokens:
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
              interleaved=True, outputs=None, stream=None):
    """sfa_norm_rope on torch CUDA tensors: normalises k (..., 1, 512) and q
    (..., N1, 512) by their weights (512,), rotates k_rope (..., 1, 64) and
    q_rope (..., N1, 64) by cos_sin[positions] (fp32 (P, 64): 32 cosines, 32
    sines).  Each of the four rows may be left out.  Returns (q, q_rope, k,
    k_rope, q_rstd, k_rstd), None where its input is; `outputs`: such a tuple
    to write into, where an output may be its own input."""
    p, lead, heads, dt, dev, pos, cs, (qa, qra, ka, kra) = _rows(q, q_rope, k, k_rope, positions, cos_sin, eps,
                                                                 interleaved)
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
    _call(dev, stream, _lib().sfa_norm_rope, "sfa_norm_rope", _pack_rows(*p), pos, cs, qa, qw, qra, ka, kw, kra, *o)
    return outputs


@_on_stream
def norm_rope_grad(positions, cos_sin, *, k=None, k_weight=None, k_rstd=None, dk=None, dk_rope=None, q=None,
                   q_weight=None, q_rstd=None, dq=None, dq_rope=None, interleaved=True, workspace=None, stream=None):
    """sfa_norm_rope_grad: gradients of norm_rope's inputs from those of its
    outputs (dq, dq_rope, dk, dk_rope, for instance sfa_grad's; where the row
    is key and value, dk is the sum of its dK and dV).  k, k_weight and k_rstd
    (q, ...) are norm_rope's inputs and its saved rstd.  Returns (dq, dq_rope,
    dk, dk_rope, dq_weight, dk_weight); the weights' gradients are fp32, summed
    in a fixed order."""
    p, lead, heads, dt, dev, pos, cs, (dqa, dqra, dka, dkra) = _rows(dq, dq_rope, dk, dk_rope, positions, cos_sin, 0.0,
                                                                     interleaved)
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
    _call(dev, stream, _lib().sfa_norm_rope_grad, "sfa_norm_rope_grad", _pack_rows(*p), pos, cs, *saved["q"],
          *saved["k"], dqa, dqra, dka, dkra, *o, ws, nbytes)
    return tuple(out)


def norm_rope_grad_workspace_size(p: RowsParams) -> int:
    n = ctypes.c_size_t(0)
    _check(_lib().sfa_norm_rope_grad_workspace_size(ctypes.byref(p), ctypes.byref(n)),
           "sfa_norm_rope_grad_workspace_size")
    return n.value


# ------------------------------------------------------------------ paged cache
def make_paged_params(cache, block_table, act_seq_kv, *, tokens, heads, layout="BSND", seq=None, act_seq_q=None,
                      scale=1.0, sparse_mode=3, interleaved=True, wait_limit_us=0) -> PagedParams:
    """Parameters of the paged calls, with checks of the cache and of the index
    tensors.  `tokens`: rows of q (B * S1 for BSND, with `seq` = S1)."""
    return PagedParams(*_paged(cache, block_table, act_seq_kv, tokens, heads, layout, seq, act_seq_q, scale,
                               sparse_mode, interleaved, wait_limit_us)[0])


def _paged(cache, block_table, act_seq_kv, tokens, heads, layout, seq, act_seq_q, scale, sparse_mode, interleaved,
           wait_limit_us):
    """The fields of PagedParams, and the addresses of cache, block_table,
    act_seq_q and act_seq_kv."""
    if cache.dtype not in DTYPES:
        raise ValueError("cache must be bfloat16 or float16")
    if cache.dim() != 3 or cache.shape[2] not in (512, 576):
        raise ValueError("cache: expected (num_pages, page_size, 576) or (num_pages, page_size, 512)")
    if block_table.dim() != 2:
        raise ValueError("block_table: expected (B, max_pages)")
    dev = cache.get_device()
    pages, page, width = cache.shape
    b, per = block_table.shape
    at = (_need("cache", cache, cache.shape, cache.dtype, dev),
          _need("block_table", block_table, block_table.shape, torch.int32, dev))
    kva = _need("act_seq_kv", act_seq_kv, (b,), torch.int32, dev)
    lay = LAYOUTS[layout.upper()]
    qla = None
    if act_seq_q is not None or lay == 1:
        qla = _need("act_seq_q", act_seq_q, (b,), torch.int32, dev)
    if lay == 0 and tokens != b * seq:
        raise ValueError(f"BSND rows of {tokens} tokens do not match {b} sequences of {seq}")
    return (lay, DTYPES[cache.dtype], b, 0 if lay else seq, tokens if lay else 0, heads, 512, width - 512, pages, page,
            per, scale, sparse_mode, 1 if interleaved else 0, wait_limit_us), at + (qla, kva)


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
                 stream=None):
    """sfa_cache_append: writes the new tokens' rows [norm(k) || rotated
    k_rope] into `cache` (num_pages, page_size, 576 or 512); k is (B, S1, 1,
    512) or (T1, 1, 512).  act_seq_kv counts the new tokens too, and their
    positions are the last of their sequences.  With q_rope (..., N1, 64) the
    same launch rotates it into q_rope_out (allocated unless given; q_rope
    itself is allowed).  `error`: optional int32 (1,) that receives a
    SFA_DEVERR_* code.  Returns (cache, q_rope_out)."""
    lead, tokens, seq = _leading("k", k, layout)
    heads = 1 if q_rope is None else q_rope.shape[-2]
    p, (ca, bta, aq, akv) = _paged(cache, block_table, act_seq_kv, tokens, heads, layout, seq, act_seq_q, 1.0, 3,
                                   interleaved, 0)
    dt, dev = cache.dtype, cache.get_device()
    ka = _need("k", k, lead + (1, 512), dt, dev)
    kw = None if k_weight is None else _need("k_weight", k_weight, (512,), dt, dev)
    kra = cs = qra = qroa = None
    table_len = 0
    if cache.shape[2] == 576:
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
    _call(dev, stream, _lib().sfa_cache_append, "sfa_cache_append", _pack_paged(*p), ca, bta, aq, akv, ka, kra, kw, eps,
          cs, table_len, qra, qroa, err)
    return cache, q_rope_out


def paged_workspace_size(p: PagedParams) -> int:
    n = ctypes.c_size_t(0)
    _check(_lib().sfa_paged_workspace_size(ctypes.byref(p), ctypes.byref(n)), "sfa_paged_workspace_size")
    return n.value


@_on_stream
def paged_fwd(q, cache, block_table, act_seq_kv, scale, *, q_rope=None, layout="BSND", act_seq_q=None, sparse_mode=3,
              out=None, softmax_max=None, softmax_sum=None, workspace=None, stream=None, wait_limit_us=0):
    """sfa_paged_fwd: attention of the new tokens' q (B, S1, N1, 512) or (T1,
    N1, 512) over their sequences' rows in the paged cache; returns (out,
    softmax_max, softmax_sum), the statistics (B, 1, S1, N1) or (1, T1, N1) as
    fwd's.  Rows of no sequence (BSND past act_seq_q, TND past the last
    sequence) are left as they were.  read_device_error reads a passed
    workspace's error word."""
    lead, tokens, seq = _leading("q", q, layout)
    heads = q.shape[-2]
    p, (ca, bta, aq, akv) = _paged(cache, block_table, act_seq_kv, tokens, heads, layout, seq, act_seq_q, scale,
                                   sparse_mode, True, wait_limit_us)
    dt, dev = cache.dtype, cache.get_device()
    qa = _need("q", q, lead + (heads, 512), dt, dev)
    qra = None
    if cache.shape[2] == 576:
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
        workspace = _workspace(paged_workspace_size(PagedParams(*p)), cache.device, workspace)
    ws = _need("workspace", workspace, workspace.shape, workspace.dtype, dev)
    _call(dev, stream, _lib().sfa_paged_fwd, "sfa_paged_fwd", _pack_paged(*p), qa, qra, ca, bta, aq, akv, oa, ma, sa, ws,
          workspace.numel() * workspace.element_size())
    return out, softmax_max, softmax_sum
