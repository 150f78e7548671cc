"""Binding of the latent-row operators (include/sfa_grad.h): the norm and
position rotation of the attention's input rows with their gradients, the
append to a paged cache, and the attention of new tokens over it.  Argument
checks and marshalling only, like the rest of the binding.
"""
from __future__ import annotations

import ctypes
from typing import Optional

import torch

from . import DTYPES, LAYOUTS, _check, _on, _ptr, _stream, _workspace, lib

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


_ready = None


def _lib():
    global _ready
    if _ready is None:
        L = lib()
        vp, sz, d, i64 = ctypes.c_void_p, ctypes.c_size_t, ctypes.c_double, ctypes.c_int64
        R, P = ctypes.POINTER(RowsParams), ctypes.POINTER(PagedParams)
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


def _need(name: str, t: Optional[torch.Tensor], shape, dtype, device):
    if t is None:
        raise ValueError(f"{name} is required")
    if t.dtype != dtype:
        raise ValueError(f"{name}: dtype {t.dtype}, expected {dtype}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name}: shape {tuple(t.shape)}, expected {tuple(shape)}")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")


# ------------------------------------------------------------------ norm and rotation
def _rows(q, q_rope, k, k_rope, positions, cos_sin, eps, interleaved):
    """Parameters, leading shape and heads from the row tensors that are there
    (queries (..., N1, 512 / 64), keys (..., 1, 512 / 64))."""
    first = next((t for t in (k, q, k_rope, q_rope) if t is not None), None)
    if first is None:
        raise ValueError("at least one of q, q_rope, k, k_rope is required")
    if first.dtype not in DTYPES:
        raise ValueError("rows must be bfloat16 or float16")
    if first.dim() < 2:
        raise ValueError("rows need a head dimension: (..., heads, 512) or (..., heads, 64)")
    lead, dev, dt = tuple(first.shape[:-2]), first.device, first.dtype
    heads = 1
    for t in (q, q_rope):
        if t is not None:
            heads = t.shape[-2]
            break
    for name, t, h, w in (("q", q, heads, 512), ("q_rope", q_rope, heads, 64), ("k", k, 1, 512),
                          ("k_rope", k_rope, 1, 64)):
        if t is not None:
            _need(name, t, lead + (h, w), dt, dev)
    tokens = 1
    for s in lead:
        tokens *= s
    if q_rope is not None or k_rope is not None:
        if positions is None or cos_sin is None:
            raise ValueError("positions and cos_sin are required with q_rope or k_rope")
    if positions is not None:
        if positions.numel() != tokens:
            raise ValueError(f"positions: {positions.numel()} elements, expected {tokens}")
        _need("positions", positions, positions.shape, torch.int32, dev)
        if cos_sin is None:
            raise ValueError("cos_sin is required with positions")
    if cos_sin is not None:
        _need("cos_sin", cos_sin, (cos_sin.shape[0], 64), torch.float32, dev)
    p = RowsParams(DTYPES[dt], 1 if interleaved else 0, tokens, heads, 0 if cos_sin is None else cos_sin.shape[0],
                   float(eps))
    return p, lead, heads, dt, dev


def norm_rope(positions, cos_sin, *, k=None, k_weight=None, k_rope=None, q=None, q_weight=None, q_rope=None, eps=1e-6,
              interleaved=True, outputs=None, stream=None):
    """sfa_norm_rope on torch CUDA tensors: normalises k (..., 1, 512) and q
    (..., N1, 512) by their weights (512,), rotates k_rope (..., 1, 64) and
    q_rope (..., N1, 64) by cos_sin[positions] (fp32 (P, 64): 32 cosines, 32
    sines).  Each of the four rows may be left out.  Returns (q, q_rope, k,
    k_rope, q_rstd, k_rstd), None where its input is; `outputs`: such a tuple
    to write into, where an output may be its own input."""
    p, lead, heads, dt, dev = _rows(q, q_rope, k, k_rope, positions, cos_sin, eps, interleaved)
    if k is not None:
        _need("k_weight", k_weight, (512,), dt, dev)
    if q is not None:
        _need("q_weight", q_weight, (512,), dt, dev)
    if outputs is None:
        outputs = (None if q is None else torch.empty_like(q), None if q_rope is None else torch.empty_like(q_rope),
                   None if k is None else torch.empty_like(k), None if k_rope is None else torch.empty_like(k_rope),
                   None if q is None else torch.empty(lead + (heads,), dtype=torch.float32, device=dev),
                   None if k is None else torch.empty(lead + (1,), dtype=torch.float32, device=dev))
    else:
        for name, o, x in zip(("q", "q_rope", "k", "k_rope"), outputs, (q, q_rope, k, k_rope)):
            if x is not None:
                _need(f"outputs: {name}", o, x.shape, dt, dev)
        for name, o, x, h in (("q_rstd", outputs[4], q, heads), ("k_rstd", outputs[5], k, 1)):
            if x is not None and o is not None:
                _need(f"outputs: {name}", o, lead + (h,), torch.float32, dev)
    qo, qro, ko, kro, rq, rk = outputs
    with _on(dev):
        _check(_lib().sfa_norm_rope(ctypes.byref(p), _ptr(positions), _ptr(cos_sin), _ptr(q), _ptr(q_weight),
                                    _ptr(q_rope), _ptr(k), _ptr(k_weight), _ptr(k_rope), _ptr(qo), _ptr(qro),
                                    _ptr(ko), _ptr(kro), _ptr(rq), _ptr(rk), _stream(stream)), "sfa_norm_rope")
    return outputs


def norm_rope_grad(positions, cos_sin, *, k=None, k_weight=None, k_rstd=None, dk=None, dk_rope=None, q=None,
                   q_weight=None, q_rstd=None, dq=None, dq_rope=None, interleaved=True, workspace=None, stream=None):
    """sfa_norm_rope_grad: gradients of norm_rope's inputs from those of its
    outputs (dq, dq_rope, dk, dk_rope, for instance sfa_grad's).  k, k_weight
    and k_rstd (q, ...) are norm_rope's inputs and its saved rstd.  Returns
    (dq, dq_rope, dk, dk_rope, dq_weight, dk_weight); the weights' gradients
    are fp32, summed in a fixed order."""
    p, lead, heads, dt, dev = _rows(dq, dq_rope, dk, dk_rope, positions, cos_sin, 0.0, interleaved)
    for name, d, x, w, r, h in (("k", dk, k, k_weight, k_rstd, 1), ("q", dq, q, q_weight, q_rstd, heads)):
        if d is not None:
            _need(name, x, d.shape, dt, dev)
            _need(f"{name}_weight", w, (512,), dt, dev)
            _need(f"{name}_rstd", r, lead + (h,), torch.float32, dev)
    gq, gqr, gk, gkr = (None if d is None else torch.empty_like(d) for d in (dq, dq_rope, dk, dk_rope))
    new = torch.empty if p.T1 else torch.zeros       # no token: the weights' gradients are empty sums
    wq = None if dq is None else new(512, dtype=torch.float32, device=dev)
    wk = None if dk is None else new(512, dtype=torch.float32, device=dev)
    if p.T1 == 0:
        return gq, gqr, gk, gkr, wq, wk
    ws, nbytes = None, 0
    with _on(dev):
        if dq is not None or dk is not None:
            ws = _workspace(norm_rope_grad_workspace_size(p), dev, workspace)
            nbytes = ws.numel() * ws.element_size()
        _check(_lib().sfa_norm_rope_grad(ctypes.byref(p), _ptr(positions), _ptr(cos_sin), _ptr(q), _ptr(q_weight),
                                         _ptr(q_rstd), _ptr(k), _ptr(k_weight), _ptr(k_rstd), _ptr(dq), _ptr(dq_rope),
                                         _ptr(dk), _ptr(dk_rope), _ptr(gq), _ptr(gqr), _ptr(gk), _ptr(gkr), _ptr(wq),
                                         _ptr(wk), _ptr(ws), nbytes, _stream(stream)), "sfa_norm_rope_grad")
    return gq, gqr, gk, gkr, wq, wk


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
    if cache.dtype not in DTYPES:
        raise ValueError("cache must be bfloat16 or float16")
    if cache.dim() != 3 or cache.shape[2] not in (512, 576):
        raise ValueError("cache: expected (num_pages, page_size, 576) or (num_pages, page_size, 512)")
    if block_table.dim() != 2:
        raise ValueError("block_table: expected (B, max_pages)")
    b, dev = block_table.shape[0], cache.device
    _need("block_table", block_table, block_table.shape, torch.int32, dev)
    _need("act_seq_kv", act_seq_kv, (b,), torch.int32, dev)
    lay = LAYOUTS[layout.upper()]
    if act_seq_q is not None or lay == 1:
        _need("act_seq_q", act_seq_q, (b,), torch.int32, dev)
    if lay == 0 and tokens != b * seq:
        raise ValueError(f"BSND rows of {tokens} tokens do not match {b} sequences of {seq}")
    return PagedParams(lay, DTYPES[cache.dtype], b, 0 if lay else seq, tokens if lay else 0, heads, 512,
                       cache.shape[2] - 512, cache.shape[0], cache.shape[1], block_table.shape[1], float(scale),
                       int(sparse_mode), 1 if interleaved else 0, int(wait_limit_us))


def _leading(name, t, layout):
    """Leading shape of rows in a layout, tokens and S1."""
    n = 2 if layout.upper() == "BSND" else 1
    if t.dim() != n + 2:
        raise ValueError(f"{name}: expected {'(B, S1' if n == 2 else '(T1'}, heads, width)")
    lead = tuple(t.shape[:n])
    tokens = lead[0] * (lead[1] if n == 2 else 1)
    return lead, tokens, lead[1] if n == 2 else None


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
    p = make_paged_params(cache, block_table, act_seq_kv, tokens=tokens, heads=heads, layout=layout, seq=seq,
                          act_seq_q=act_seq_q, interleaved=interleaved)
    dt, dev = cache.dtype, cache.device
    _need("k", k, lead + (1, 512), dt, dev)
    if k_weight is not None:
        _need("k_weight", k_weight, (512,), dt, dev)
    table_len = 0
    if p.Dr == 64:
        _need("k_rope", k_rope, lead + (1, 64), dt, dev)
        if cos_sin is None:
            raise ValueError("cos_sin is required")
        _need("cos_sin", cos_sin, (cos_sin.shape[0], 64), torch.float32, dev)
        table_len = cos_sin.shape[0]
        if q_rope is not None:
            _need("q_rope", q_rope, lead + (heads, 64), dt, dev)
            if q_rope_out is None:
                q_rope_out = torch.empty_like(q_rope)
            _need("q_rope_out", q_rope_out, lead + (heads, 64), dt, dev)
    elif k_rope is not None or q_rope is not None:
        raise ValueError("rope rows given for a cache without them")
    if error is not None:
        _need("error", error, (1,), torch.int32, dev)
    with _on(dev):
        _check(_lib().sfa_cache_append(ctypes.byref(p), _ptr(cache), _ptr(block_table), _ptr(act_seq_q),
                                       _ptr(act_seq_kv), _ptr(k), _ptr(k_rope), _ptr(k_weight), float(eps),
                                       _ptr(cos_sin), table_len, _ptr(q_rope), _ptr(q_rope_out), _ptr(error),
                                       _stream(stream)), "sfa_cache_append")
    return cache, q_rope_out


def paged_workspace_size(p: PagedParams) -> int:
    n = ctypes.c_size_t(0)
    _check(_lib().sfa_paged_workspace_size(ctypes.byref(p), ctypes.byref(n)), "sfa_paged_workspace_size")
    return n.value


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
    p = make_paged_params(cache, block_table, act_seq_kv, tokens=tokens, heads=heads, layout=layout, seq=seq,
                          act_seq_q=act_seq_q, scale=scale, sparse_mode=sparse_mode, wait_limit_us=wait_limit_us)
    dt, dev = cache.dtype, cache.device
    _need("q", q, lead + (heads, 512), dt, dev)
    if p.Dr == 64:
        _need("q_rope", q_rope, lead + (heads, 64), dt, dev)
    elif q_rope is not None:
        raise ValueError("q_rope given for a cache without rope rows")
    st_shape = (lead[0], 1, lead[1], heads) if seq is not None else (1, tokens, heads)
    if out is None:
        out = torch.empty_like(q)
    if softmax_max is None:
        softmax_max = torch.empty(st_shape, dtype=torch.float32, device=dev)
    if softmax_sum is None:
        softmax_sum = torch.empty(st_shape, dtype=torch.float32, device=dev)
    _need("out", out, q.shape, dt, dev)
    _need("softmax_max", softmax_max, st_shape, torch.float32, dev)
    _need("softmax_sum", softmax_sum, st_shape, torch.float32, dev)
    with _on(dev):
        ws = _workspace(paged_workspace_size(p), dev, workspace)
        _check(_lib().sfa_paged_fwd(ctypes.byref(p), _ptr(q), _ptr(q_rope), _ptr(cache), _ptr(block_table),
                                    _ptr(act_seq_q), _ptr(act_seq_kv), _ptr(out), _ptr(softmax_max),
                                    _ptr(softmax_sum), _ptr(ws), ws.numel() * ws.element_size(), _stream(stream)),
               "sfa_paged_fwd")
    return out, softmax_max, softmax_sum
