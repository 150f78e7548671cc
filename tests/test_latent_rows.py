"""Norm and rotation of the attention's input rows, their gradients, and the
append to the paged cache, against plain 64-bit forms."""
import ctypes

import pytest
import torch

import sfa_grad_gb300 as sfa
from latent_util import DTYPES, U32, floor_of, half_step, norm, rotate, table

EPS = 1e-6


def _rows(tokens, heads, dtype, seed=0, device="cuda", lead=None):
    g = torch.Generator().manual_seed(seed)
    t = DTYPES[dtype]
    lead = (tokens,) if lead is None else lead
    r = lambda *s: torch.randn(*s, generator=g).to(t).to(device)  # noqa: E731
    pos = torch.randint(0, 500, lead, generator=g, dtype=torch.int32)
    return dict(k=r(*lead, 1, 512) * 3, k_rope=r(*lead, 1, 64), q=r(*lead, heads, 512), q_rope=r(*lead, heads, 64),
                k_weight=r(512), q_weight=r(512), positions=pos.to(device), cs=table(500, device))


def _close(got, ref, bound, what):
    err = (got.double() - ref).abs()
    assert bool((err <= bound).all()), f"{what}: worst excess {float((err - bound).max()):.3e}"


def _turn_bound(x, ref):
    # two products and a sum in fp32 (3 units of |a| + |b|), one rounding to the type
    return half_step(x.dtype) * 1.01 * ref.abs() + 6 * U32 * x.double().abs().amax(-1, keepdim=True) + floor_of(x.dtype)


def _norm_bound(x, ref):
    # the mean of squares adds 16 terms a lane and 5 levels of lanes (all
    # positive), the root halves that; two more products
    return (half_step(x.dtype) * 1.01 + 24 * U32) * ref.abs() + floor_of(x.dtype)


# ------------------------------------------------------------------ refusals (CPU)
def test_row_refusals():
    x = _rows(3, 2, "bf16", device="cpu")
    ok = dict(k=x["k"], k_weight=x["k_weight"])
    for kw, what in (
            (dict(), "at least one"),
            (dict(k=x["k"]), "k_weight is required"),
            (dict(q=x["q"], q_weight=x["q_weight"][:256]), "q_weight: shape"),
            (dict(ok, k_weight=x["k_weight"].float()), "k_weight: dtype"),
            (dict(k=x["k"].float(), k_weight=x["k_weight"]), "bfloat16 or float16"),
            (dict(ok, q_rope=x["q_rope"][:2]), "q_rope: shape"),
            (dict(ok, k_rope=x["k_rope"].half()), "k_rope: dtype")):
        with pytest.raises(ValueError, match=what):
            sfa.norm_rope(x["positions"], x["cs"], **kw)
    with pytest.raises(ValueError, match="positions and cos_sin"):
        sfa.norm_rope(None, None, k_rope=x["k_rope"])
    with pytest.raises(ValueError, match="positions: 3"):
        sfa.norm_rope(x["positions"], x["cs"], k_rope=x["k_rope"][:2])
    with pytest.raises(ValueError, match="positions: dtype"):
        sfa.norm_rope(x["positions"].long(), x["cs"], k_rope=x["k_rope"])
    with pytest.raises(ValueError, match="cos_sin: shape"):
        sfa.norm_rope(x["positions"], x["cs"][:, :32], k_rope=x["k_rope"])
    with pytest.raises(ValueError, match="(?i)cuda device"):
        sfa.norm_rope(x["positions"], x["cs"], **ok)
    with pytest.raises(ValueError, match="k_rstd is required"):
        sfa.norm_rope_grad(None, None, k=x["k"], k_weight=x["k_weight"], dk=x["k"])


def _c_rows(**over):
    from sfa_grad_gb300.latent import RowsParams
    d = dict(dtype=0, interleaved=1, T1=4, N1=2, table_len=10, eps=1e-6)
    d.update(over)
    return RowsParams(*d.values())


def test_row_codes():
    from sfa_grad_gb300.latent import _lib
    n = ctypes.c_size_t(0)
    size = lambda p: _lib().sfa_norm_rope_grad_workspace_size(ctypes.byref(p), ctypes.byref(n))  # noqa: E731
    assert size(_c_rows()) == 0 and n.value >= 2 * 2048
    assert _lib().sfa_norm_rope_grad_workspace_size(None, ctypes.byref(n)) == sfa.SFA_ERR_NULLPTR
    for over in (dict(N1=0), dict(N1=129), dict(T1=-1), dict(T1=1 << 31), dict(T1=1 << 29, N1=128),
                 dict(eps=float("nan")), dict(eps=-1.0), dict(table_len=-1)):
        assert size(_c_rows(**over)) == sfa.SFA_ERR_SHAPE, over
    for over in (dict(dtype=2), dict(interleaved=2)):
        assert size(_c_rows(**over)) == sfa.SFA_ERR_PARAM_INVALID, over
    fake, odd = ctypes.c_void_p(16), ctypes.c_void_p(24)
    call = lambda p, *a: _lib().sfa_norm_rope(ctypes.byref(p), *a)  # noqa: E731
    # order: positions, cos_sin, q, qw, qr, k, kw, kr, four outputs, two rstd, stream
    none = [None] * 15
    assert call(_c_rows(), *none[:5], fake, *none[6:]) == sfa.SFA_ERR_NULLPTR               # k without weight
    a = list(none); a[4] = a[9] = fake
    assert call(_c_rows(), *a) == sfa.SFA_ERR_NULLPTR                                         # rope without table
    a[0] = a[1] = fake
    assert call(_c_rows(table_len=0), *a) == sfa.SFA_ERR_SHAPE
    a[4] = odd
    assert call(_c_rows(), *a) == sfa.SFA_ERR_PARAM_INVALID                                   # misaligned
    g = [None] * 18 + [None, 0, None]
    g[5] = g[6] = g[7] = g[10] = g[14] = g[17] = fake                                          # k, kw, rstd, d_k, dk, dkw
    grad = lambda *a: _lib().sfa_norm_rope_grad(ctypes.byref(_c_rows()), *a)  # noqa: E731
    assert grad(*g) == sfa.SFA_ERR_NULLPTR                                                     # no workspace
    g[18], g[19] = ctypes.c_void_p(256), 8
    assert grad(*g) == sfa.SFA_ERR_PARAM_INVALID                                               # short workspace


# ------------------------------------------------------------------ norm and rotation
@pytest.mark.gpu
@pytest.mark.parametrize("tokens,heads,dtype,inter", [
    (1, 1, "bf16", True), (7, 128, "bf16", True), (33, 16, "fp16", False), (130, 3, "bf16", False),
    (5, 17, "fp16", True), (1000, 48, "bf16", False)])
def test_norm_rope(tokens, heads, dtype, inter):
    x = _rows(tokens, heads, dtype)
    x["positions"][::5] = -1                      # padding
    x["positions"][3::7] = 500
    pad = (x["positions"] < 0) | (x["positions"] >= 500)
    q, qr, k, kr, rq, rk = sfa.norm_rope(x["positions"], x["cs"], k=x["k"], k_weight=x["k_weight"],
                                         k_rope=x["k_rope"], q=x["q"], q_weight=x["q_weight"], q_rope=x["q_rope"],
                                         eps=EPS, interleaved=inter)
    for name, got, rstd, src, w in (("k", k, rk, x["k"], x["k_weight"]), ("q", q, rq, x["q"], x["q_weight"])):
        y, r = norm(src, w, EPS)
        y[pad], r[pad] = 0, 0
        _close(got, y, _norm_bound(src, y), name)
        _close(rstd, r, 24 * U32 * r, name + " rstd")
    for name, got, src in (("k_rope", kr, x["k_rope"]), ("q_rope", qr, x["q_rope"])):
        y = rotate(src, x["cs"], x["positions"], inter)
        _close(got, y, _turn_bound(src, y), name)


@pytest.mark.gpu
def test_norm_rope_partial_and_in_place():
    """Each row alone; outputs over the inputs; BSND leading shape; no position
    needed for norms alone; values of 1e4 and an all-zero row."""
    x = _rows(6, 4, "bf16", lead=(2, 3))
    both = sfa.norm_rope(x["positions"], x["cs"], k=x["k"], k_weight=x["k_weight"], k_rope=x["k_rope"],
                         q_rope=x["q_rope"], interleaved=False)
    assert both[0] is None and both[4] is None and both[5].shape == (2, 3, 1)
    alone = sfa.norm_rope(None, None, k=x["k"], k_weight=x["k_weight"])
    assert torch.equal(alone[2], both[2])
    turned = sfa.norm_rope(x["positions"], x["cs"], q_rope=x["q_rope"], interleaved=False)[1]
    assert torch.equal(turned, both[1])
    kr, qr, k = x["k_rope"].clone(), x["q_rope"].clone(), x["k"].clone()
    sfa.norm_rope(x["positions"], x["cs"], k=k, k_weight=x["k_weight"], k_rope=kr, q_rope=qr, interleaved=False,
                  outputs=(None, qr, k, kr, None, None))
    assert torch.equal(k, both[2]) and torch.equal(qr, both[1]) and torch.equal(kr, both[3])
    z = torch.zeros(2, 1, 512, dtype=torch.bfloat16, device="cuda")
    z[1] = 1e4
    y = sfa.norm_rope(None, None, k=z, k_weight=x["k_weight"])[2]
    assert not y[0].any()
    assert torch.equal(y[1, 0], x["k_weight"])     # x / rms = 1 within half a step
    e = torch.empty(0, 1, 512, dtype=torch.bfloat16, device="cuda")
    assert sfa.norm_rope(None, None, k=e, k_weight=x["k_weight"])[2].shape == (0, 1, 512)


# ------------------------------------------------------------------ gradients
def _grad_ref(x, w, r, dy, pad):
    x, w, r, dy = x.double(), w.double(), r.double(), dy.double()
    dy = torch.where(pad[:, None, None], 0.0, dy)
    xh = x * r[..., None]
    g = dy * w
    c = (g * xh).mean(-1, keepdim=True)
    dx = r[..., None] * (g - xh * c)
    size = r[..., None] * (g.abs() + xh.abs() * (g * xh).abs().mean(-1, keepdim=True))
    return dx, size, (dy * xh).flatten(0, 1).sum(0), (dy * xh).abs().flatten(0, 1).sum(0)


@pytest.mark.gpu
@pytest.mark.parametrize("tokens,heads,dtype,inter", [
    (1, 1, "bf16", True), (37, 16, "fp16", False), (300, 3, "bf16", True), (9, 128, "fp16", True),
    (4100, 2, "bf16", False)])
def test_norm_rope_grad(tokens, heads, dtype, inter):
    x, d = _rows(tokens, heads, dtype), _rows(tokens, heads, dtype, seed=1)
    x["positions"][2::6] = -3
    pad = x["positions"] < 0
    fw = sfa.norm_rope(x["positions"], x["cs"], k=x["k"], k_weight=x["k_weight"], q=x["q"], q_weight=x["q_weight"])
    args = dict(k=x["k"], k_weight=x["k_weight"], k_rstd=fw[5], dk=d["k"], dk_rope=d["k_rope"], q=x["q"],
                q_weight=x["q_weight"], q_rstd=fw[4], dq=d["q"], dq_rope=d["q_rope"], interleaved=inter)
    out = sfa.norm_rope_grad(x["positions"], x["cs"], **args)
    dq, dqr, dk, dkr, wq, wk = out
    u = half_step(DTYPES[dtype])
    for name, got, gw, src, w, r, dy in (("k", dk, wk, x["k"], x["k_weight"], fw[5], d["k"]),
                                         ("q", dq, wq, x["q"], x["q_weight"], fw[4], d["q"])):
        ref, size, rw, aw = _grad_ref(src, w, r, dy, pad)
        # the mean: 16 terms a lane, 5 levels; a few products on top
        _close(got, ref, 1.01 * u * ref.abs() + 32 * U32 * size + floor_of(src.dtype), "d" + name)
        # sums in chains of at most all rows, then of partial sums
        _close(gw, rw, (min(src.shape[0] * src.shape[1], 400) + 16) * U32 * aw, f"d{name}_weight")
    for name, got, dy in (("dk_rope", dkr, d["k_rope"]), ("dq_rope", dqr, d["q_rope"])):
        ref = rotate(dy, x["cs"], x["positions"], inter, back=True)
        _close(got, ref, _turn_bound(dy, ref), name)
    again = sfa.norm_rope_grad(x["positions"], x["cs"], **args)
    assert all(torch.equal(a, b) for a, b in zip(out, again))
    only = sfa.norm_rope_grad(None, None, k=x["k"], k_weight=x["k_weight"], k_rstd=fw[5], dk=d["k"]) \
        if not pad.any() else None
    assert only is None or torch.equal(only[2], dk)


@pytest.mark.gpu
def test_norm_rope_grad_differences():
    """The gradients against central differences of the 64-bit forward."""
    x, d = _rows(2, 2, "fp16", seed=3), _rows(2, 2, "fp16", seed=4)

    def loss(k, kr, w):
        y, _ = norm(k, w, EPS)
        return (y * d["k"].double()).sum() + (rotate(kr, x["cs"], x["positions"], True) * d["k_rope"].double()).sum()

    fw = sfa.norm_rope(x["positions"], x["cs"], k=x["k"], k_weight=x["k_weight"])
    _, _, dk, dkr, _, wk = sfa.norm_rope_grad(x["positions"], x["cs"], k=x["k"], k_weight=x["k_weight"],
                                              k_rstd=fw[5], dk=d["k"], dk_rope=d["k_rope"])
    base = [x["k"].double(), x["k_rope"].double(), x["k_weight"].double()]
    h = 1e-4
    for which, got, places in ((0, dk, [(0, 0, 0), (1, 0, 511), (1, 0, 77)]), (1, dkr, [(0, 0, 0), (1, 0, 63)]),
                               (2, wk, [(0,), (300,)])):
        for at in places:
            up, dn = [t.clone() for t in base], [t.clone() for t in base]
            up[which][at] += h
            dn[which][at] -= h
            diff = float((loss(*up) - loss(*dn)) / (2 * h))
            # h^2 of the third derivative (values of a few units) and the output's rounding
            assert abs(float(got[at]) - diff) <= half_step(torch.float16) * 1.1 * abs(diff) + 1e-5


@pytest.mark.gpu
def test_norm_rope_grad_empty():
    e = torch.empty(0, 1, 512, dtype=torch.bfloat16, device="cuda")
    w = torch.ones(512, dtype=torch.bfloat16, device="cuda")
    r = torch.empty(0, 1, device="cuda")
    out = sfa.norm_rope_grad(None, None, k=e, k_weight=w, k_rstd=r, dk=e)
    assert out[2].shape == e.shape and not out[5].any()


@pytest.mark.gpu
def test_norm_rope_grad_captured():
    """Captured and replayed on new gradients, with its own workspace."""
    x, d = _rows(50, 8, "bf16"), _rows(50, 8, "bf16", seed=5)
    fw = sfa.norm_rope(x["positions"], x["cs"], k=x["k"], k_weight=x["k_weight"])
    ws = torch.empty(1 << 22, dtype=torch.uint8, device="cuda")
    call = lambda dk: sfa.norm_rope_grad(x["positions"], x["cs"], k=x["k"], k_weight=x["k_weight"], k_rstd=fw[5],  # noqa: E731
                                         dk=dk, dk_rope=d["k_rope"], workspace=ws)
    buf = d["k"].clone()
    call(buf)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = call(buf)
    buf.mul_(-2)
    g.replay()
    want = call(buf)
    torch.cuda.synchronize()
    assert torch.equal(out[2], want[2]) and torch.equal(out[5], want[5])


# ------------------------------------------------------------------ append
def _append_case(qlens, kvlens, heads, dtype, page, layout="TND", s1=None, extra=0, width=576, seed=0):
    g = torch.Generator().manual_seed(seed)
    t = DTYPES[dtype]
    need = [-(-max(k, 1) // page) for k in kvlens]
    pages = sum(need) + 2
    order = torch.randperm(pages, generator=g).int()
    bt = torch.full((len(kvlens), max(need) + 1), -7, dtype=torch.int32)
    at = 0
    for b, n in enumerate(need):
        bt[b, :n] = order[at:at + n]
        at += n
    lead = (len(qlens), s1) if layout == "BSND" else (sum(qlens) + extra,)
    r = lambda *s: torch.randn(*s, generator=g).to(t).cuda()  # noqa: E731
    return dict(cache=r(pages, page, width), bt=bt.cuda(), aq=torch.tensor(qlens, dtype=torch.int32).cuda(),
                akv=torch.tensor(kvlens, dtype=torch.int32).cuda(), k=r(*lead, 1, 512), k_rope=r(*lead, 1, 64),
                q_rope=r(*lead, heads, 64), w=r(512), cs=table(600, "cuda"))


def _append_ref(x, qlens, kvlens, layout, inter, normed):
    """The cache and rotated queries in 64 bits, with bounds (zero where
    nothing may change)."""
    page = x["cache"].shape[1]
    cache, bound = x["cache"].double().flatten(0, 1), torch.zeros_like(x["cache"], dtype=torch.float64).flatten(0, 1)
    qr = torch.full_like(x["q_rope"], 9.0, dtype=torch.float64)
    qb = torch.zeros_like(qr)
    first = 0
    for b, (a, m) in enumerate(zip(qlens, kvlens)):
        rows = (slice(first, first + a),) if layout == "TND" else (b, slice(0, a))
        first += a
        pos = torch.arange(m - a, m, device="cuda")
        at = x["bt"][b][pos // page].long() * page + pos % page
        k = x["k"][rows]
        y = norm(k, x["w"], EPS)[0][:, 0] if normed else k.double()[:, 0]
        cache[at, :512] = y
        bound[at, :512] = _norm_bound(k, y) if normed else 0.0
        if cache.shape[1] == 576:
            y = rotate(x["k_rope"][rows], x["cs"], pos, inter)
            cache[at, 512:], bound[at, 512:] = y[:, 0], _turn_bound(x["k_rope"][rows], y)[:, 0]
            y = rotate(x["q_rope"][rows], x["cs"], pos, inter)
            qr[rows], qb[rows] = y, _turn_bound(x["q_rope"][rows], y)
    return cache.view(x["cache"].shape), bound.view(x["cache"].shape), qr, qb


@pytest.mark.gpu
@pytest.mark.parametrize("qlens,kvlens,heads,dtype,page,layout,inter,normed", [
    ([1], [1], 1, "bf16", 16, "BSND", True, True),
    ([1] * 70, list(range(1, 71)), 16, "bf16", 64, "TND", True, True),
    ([3, 0, 40, 1], [3, 0, 333, 129], 128, "fp16", 48, "TND", False, True),
    ([17, 5, 0], [17, 500, 64], 3, "bf16", 128, "BSND", False, False),
    ([0] * 60 + [4] + [0] * 9 + [70], [0] * 60 + [600] + [5] * 9 + [70], 17, "fp16", 1024, "TND", True, True)])
def test_append(qlens, kvlens, heads, dtype, page, layout, inter, normed):
    s1 = max(qlens) if layout == "BSND" else None
    x = _append_case(qlens, kvlens, heads, dtype, page, layout, s1, extra=5 if layout == "TND" else 0)
    want, bound, qr, qb = _append_ref(x, qlens, kvlens, layout, inter, normed)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = torch.full_like(x["q_rope"], 9.0)
    sfa.cache_append(x["cache"], x["bt"], x["akv"], x["k"], x["k_rope"], x["cs"], k_weight=x["w"] if normed else None,
                     eps=EPS, interleaved=inter, q_rope=x["q_rope"], q_rope_out=out, layout=layout,
                     act_seq_q=x["aq"], error=err)
    _close(x["cache"], want, bound, "cache")
    _close(out, qr, qb, "q_rope")
    assert int(err) == 0


@pytest.mark.gpu
def test_append_without_rope_and_in_place():
    x = _append_case([2, 2], [2, 90], 4, "bf16", 32, "BSND", 2, width=512)
    want, bound, _, _ = _append_ref(x, [2, 2], [2, 90], "BSND", True, True)
    sfa.cache_append(x["cache"], x["bt"], x["akv"], x["k"], k_weight=x["w"], eps=EPS)
    _close(x["cache"], want, bound, "cache")
    x = _append_case([2, 2], [2, 90], 4, "bf16", 32, "BSND", 2)
    _, _, qr, qb = _append_ref(x, [2, 2], [2, 90], "BSND", True, True)
    sfa.cache_append(x["cache"], x["bt"], x["akv"], x["k"], x["k_rope"], x["cs"], q_rope=x["q_rope"],
                     q_rope_out=x["q_rope"])
    _close(x["q_rope"], qr, qb, "q_rope in place")


@pytest.mark.gpu
@pytest.mark.parametrize("what,code", [("page", 3), ("negative page", 3), ("position", 4), ("kv long", 2),
                                       ("kv short", 2), ("negative q", 2)])
def test_append_leaves_out(what, code):
    """A token that cannot be placed is left out and reported; the others are written."""
    qlens, kvlens = [2, 1], [40, 30]
    x = _append_case(qlens, kvlens, 2, "bf16", 16)
    if what == "page":
        x["bt"][1, 1] = x["cache"].shape[0]
    elif what == "negative page":
        x["bt"][1, 1] = -1
    elif what == "position":
        x["cs"] = x["cs"][:29].contiguous()
        x["akv"][0] = kvlens[0] = 20
    elif what == "kv long":
        x["akv"][1] = x["bt"].shape[1] * 16 + 1
    elif what == "kv short":
        x["akv"][1] = 0
    else:
        x["aq"][1] = -1
    want, bound, qr, qb = _append_ref(x, qlens[:1], kvlens[:1], "TND", True, True)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = torch.full_like(x["q_rope"], 9.0)
    sfa.cache_append(x["cache"], x["bt"], x["akv"], x["k"], x["k_rope"], x["cs"], k_weight=x["w"], eps=EPS,
                     q_rope=x["q_rope"], q_rope_out=out, layout="TND", act_seq_q=x["aq"], error=err)
    _close(x["cache"], want, bound, "cache")
    _close(out[:2], qr[:2], qb[:2], "q_rope")
    assert int(err) == code
