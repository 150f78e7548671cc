"""Attention of new tokens over the paged latent cache, against a plain 64-bit
form, and the whole serving step (append, attention) against the framework's
forward over contiguous rows."""
import ctypes

import pytest
import torch

import sfa_grad_gb300 as sfa
from latent_util import DTYPES, U32, paged_inputs, paged_ref, table

SCALE = 576 ** -0.5
UNTOUCHED = 7.0


def _call(x, scale=SCALE, mode=3, layout="TND", **kw):
    return sfa.paged_fwd(x["q"], x["cache"], x["block_table"], x["act_seq_kv"], scale, q_rope=x["q_rope"],
                         layout=layout, act_seq_q=x["act_seq_q"], sparse_mode=mode, **kw)


def _buffers(x):
    q = x["q"]
    st = (1, q.shape[0], q.shape[1]) if q.dim() == 3 else (q.shape[0], 1, q.shape[1], q.shape[2])
    return dict(out=torch.full_like(q, UNTOUCHED), softmax_max=torch.full(st, UNTOUCHED, device="cuda"),
                softmax_sum=torch.full(st, UNTOUCHED, device="cuda"))


def _check(x, got, qlens, kvlens, scale=SCALE, mode=3, layout="TND"):
    out, smax, ssum = got
    smax, ssum = smax.view(out.shape[:-1]), ssum.view(out.shape[:-1])
    mine = torch.zeros(out.shape[:-1], dtype=torch.bool, device="cuda")
    for rows, o, m, l, (bo, bm, bl) in paged_ref(x, qlens, kvlens, scale, mode, layout):
        mine[rows] = True
        none = l == 0
        assert torch.equal(smax[rows].double() == -float("inf"), none)
        for name, a, b, bound in (("out", out[rows].double(), o, bo),
                                  ("max", smax[rows].double()[~none], m[~none], bm[~none]),
                                  ("sum", ssum[rows].double(), l, bl * l)):
            err = (a - b).abs()
            assert bool((err <= bound).all()), f"{name} {rows}: worst excess {float((err - bound).max()):.3e}"
    for t in got:
        left = t.view(*out.shape[:-1], -1)[~mine]
        assert bool((left == UNTOUCHED).all()), "rows of no sequence were written"


CASES = {
    # qlens, kvlens, heads, dtype, page, rope, mode, layout, s1, extra
    "one_key": ([1], [1], 1, "bf16", 16, True, 3, "BSND", 1, 0),
    "no_key": ([1, 2, 3], [0, 1, 0], 4, "fp16", 16, True, 3, "TND", None, 0),
    "more_new_than_cached": ([5, 200], [3, 150], 16, "bf16", 32, True, 3, "TND", None, 0),
    "borders": ([1] * 9, [63, 64, 65, 127, 128, 129, 255, 256, 257], 16, "bf16", 64, True, 3, "TND", None, 3),
    "heads_3": ([1, 7, 50], [900, 300, 50], 3, "fp16", 48, True, 3, "TND", None, 0),
    "heads_128": ([1, 2, 1], [1000, 130, 17], 128, "bf16", 64, True, 3, "TND", None, 2),
    "heads_128_chunk": ([70], [700], 128, "bf16", 128, True, 3, "TND", None, 0),
    "heads_64_chunk": ([33, 1, 0, 20], [133, 64, 99, 1020], 64, "fp16", 16, True, 3, "TND", None, 0),
    "heads_48": ([9, 4], [300, 77], 48, "bf16", 256, True, 3, "BSND", 12, 0),
    "heads_100": ([3], [400], 100, "bf16", 1024, True, 3, "TND", None, 0),
    "no_mask": ([5, 40], [200, 40], 24, "bf16", 64, True, 0, "TND", None, 0),
    "no_mask_short": ([9, 3], [4, 0], 2, "bf16", 64, True, 0, "TND", None, 0),
    "no_rope": ([2, 20], [500, 129], 32, "bf16", 64, False, 3, "TND", None, 0),
    "no_rope_128": ([2], [300], 128, "fp16", 32, False, 3, "BSND", 3, 0),
    "many": ([0, 1, 2] * 100, [37 * (i % 11) + 2 for i in range(300)], 8, "bf16", 16, True, 3, "TND", None, 5),
    "long_16": ([1], [20011], 16, "bf16", 64, True, 3, "TND", None, 0),
    "long_128": ([2], [9001], 128, "fp16", 64, True, 3, "TND", None, 0),
    "long_chunk_6": ([300, 1], [4500, 3000], 6, "bf16", 64, True, 3, "TND", None, 0),
}


def _inputs(name, **kw):
    qlens, kvlens, heads, dtype, page, rope, mode, layout, s1, extra = CASES[name]
    x = paged_inputs(qlens, kvlens, heads, dtype, page=page, rope=rope, layout=layout, s1=s1, extra=extra, **kw)
    return x, qlens, kvlens, mode, layout


# ------------------------------------------------------------------ refusals (CPU)
def _params(**over):
    from sfa_grad_gb300.latent import PagedParams
    d = dict(layout=1, dtype=0, B=2, S1=0, T1=4, N1=16, D=512, Dr=64, num_pages=8, page_size=64, max_pages=4,
             scale=1.0, sparse_mode=3, interleaved=1, wait_limit_us=0)
    d.update(over)
    return PagedParams(*d.values())


def test_paged_codes():
    from sfa_grad_gb300.latent import _lib
    n = ctypes.c_size_t(0)
    size = lambda p: _lib().sfa_paged_workspace_size(ctypes.byref(p), ctypes.byref(n))  # noqa: E731
    assert size(_params()) == 0 and n.value >= 4
    for over in (dict(D=256), dict(Dr=32), dict(N1=0), dict(N1=129), dict(B=0), dict(page_size=8),
                 dict(page_size=72), dict(page_size=2048), dict(num_pages=0), dict(num_pages=1 << 30),
                 dict(max_pages=0), dict(sparse_mode=1), dict(scale=float("inf")), dict(T1=-1), dict(T1=1 << 31),
                 dict(layout=0, S1=1 << 24, B=1 << 10)):
        assert size(_params(**over)) == sfa.SFA_ERR_SHAPE, over
    for over in (dict(dtype=3), dict(layout=2), dict(interleaved=-1), dict(wait_limit_us=-1)):
        assert size(_params(**over)) == sfa.SFA_ERR_PARAM_INVALID, over
    assert _lib().sfa_paged_workspace_size(None, ctypes.byref(n)) == sfa.SFA_ERR_NULLPTR
    f = ctypes.c_void_p(256)
    call = lambda p, a, b: _lib().sfa_paged_fwd(ctypes.byref(p), *a, b, None)  # noqa: E731
    for i in (0, 1, 2, 3, 4, 5, 6, 7, 8, 9):            # q, q_rope, cache, table, lengths, outputs, workspace
        a = [f] * 10
        a[i] = None
        assert call(_params(), a, 1 << 40) == sfa.SFA_ERR_NULLPTR, i
    assert call(_params(), [f] * 10, 1) == sfa.SFA_ERR_PARAM_INVALID
    a = [f] * 10
    a[0] = ctypes.c_void_p(8)
    assert call(_params(), a, 1 << 40) == sfa.SFA_ERR_PARAM_INVALID
    app = lambda p, a: _lib().sfa_cache_append(ctypes.byref(p), *a)  # noqa: E731
    # cache, table, act q, act kv, k, k_rope, weight, eps, cos_sin, table_len, q_rope, out, error, stream
    ok = [f, f, f, f, f, f, None, 1e-6, f, 9, None, None, None, None]
    for i in (0, 1, 2, 3, 4, 5, 8):
        a = list(ok)
        a[i] = None
        assert app(_params(), a) == sfa.SFA_ERR_NULLPTR, i
    a = list(ok); a[9] = 0
    assert app(_params(), a) == sfa.SFA_ERR_SHAPE
    a = list(ok); a[10] = f
    assert app(_params(), a) == sfa.SFA_ERR_NULLPTR


def test_paged_refusals():
    x = paged_inputs([2, 1], [20, 5], 4, "bf16", page=16, device="cpu")

    def refused(match, **over):
        y = dict(x, **over)
        with pytest.raises(ValueError, match=match):
            _call(y)

    refused("cache must be", cache=x["cache"].float())
    refused("cache: expected", cache=x["cache"][..., :500])
    refused("block_table: expected", block_table=x["block_table"][0])
    refused("block_table: dtype", block_table=x["block_table"].long())
    refused("act_seq_kv: shape", act_seq_kv=x["act_seq_kv"][:1])
    refused("act_seq_q is required", act_seq_q=None)
    refused("q: dtype", q=x["q"].half())
    refused("q: shape", q=x["q"][..., :256])
    refused("q_rope: shape", q_rope=x["q_rope"][:2])
    refused("q_rope is required", q_rope=None)
    refused("(?i)cuda device")
    with pytest.raises(ValueError, match="out: shape"):
        _call(x, out=x["q"][:1])
    with pytest.raises(ValueError, match="BSND rows"):
        _call(dict(x, q=x["q"][None], q_rope=x["q_rope"][None]), layout="BSND")
    with pytest.raises(ValueError, match="rope rows given"):
        sfa.cache_append(x["cache"][..., :512].contiguous(), x["block_table"], x["act_seq_kv"],
                         x["q"][:, :1].contiguous(), x["q_rope"][:, :1].contiguous(), layout="TND",
                         act_seq_q=x["act_seq_q"])


# ------------------------------------------------------------------ against 64 bits
@pytest.mark.gpu
@pytest.mark.parametrize("name", list(CASES))
def test_paged(name):
    x, qlens, kvlens, mode, layout = _inputs(name)
    got = _call(x, mode=mode, layout=layout, **_buffers(x))
    torch.cuda.synchronize()
    _check(x, got, qlens, kvlens, mode=mode, layout=layout)


@pytest.mark.gpu
@pytest.mark.parametrize("name", ["heads_3", "heads_128", "long_16"])
@pytest.mark.parametrize("scale", [0.7, -SCALE, 0.0])
def test_paged_scales(name, scale):
    """Peaked, reversed and flat distributions."""
    x, qlens, kvlens, mode, layout = _inputs(name, q_scale=0.5)
    _check(x, _call(x, scale=scale, mode=mode, layout=layout, **_buffers(x)), qlens, kvlens, scale, mode, layout)


@pytest.mark.gpu
@pytest.mark.parametrize("heads,dtype", [(16, "bf16"), (128, "fp16")])
def test_paged_rising_scores(heads, dtype):
    """Scores that rise along the sequence by hundreds: the running max moves
    at every tile."""
    x = paged_inputs([1, 3], [1500, 700], heads, dtype, seed=4)
    d = torch.randn(576, generator=torch.Generator().manual_seed(9)).cuda()
    d /= d.norm()
    for b, m in enumerate([1500, 700]):
        j = torch.arange(m, device="cuda")
        rows = x["block_table"][b][j // 64].long() * 64 + j % 64
        flat = x["cache"].view(-1, 576)
        flat[rows] = (flat[rows].float() * 0.1 + (j / m * 24)[:, None] * d).to(flat.dtype)
    full = 24 * d * 1.0
    x["q"][:] = (x["q"].float() * 0.1 + full[:512]).to(x["q"].dtype)
    x["q_rope"][:] = (x["q_rope"].float() * 0.1 + full[512:]).to(x["q"].dtype)
    _check(x, _call(x, scale=0.5, **_buffers(x)), [1, 3], [1500, 700], 0.5)


@pytest.mark.gpu
@pytest.mark.parametrize("heads", [16, 128])
def test_paged_nan_ahead(heads):
    """NaN and infinities in a later token's row do not reach earlier tokens."""
    x = paged_inputs([6], [200], heads, "bf16")
    clean = _call(x, **_buffers(x))[0].clone()
    flat = x["cache"].view(-1, 576)
    for at, v in ((199, float("nan")), (198, float("inf"))):
        flat[x["block_table"][0, at // 64].long() * 64 + at % 64] = v
    out = _call(x, **_buffers(x))[0]
    assert torch.equal(out[:4], clean[:4])
    assert bool(out[5].isnan().any())


@pytest.mark.gpu
def test_paged_same_bits_streams_and_graph():
    """Two calls give the same bits; so does another stream; a graph captured
    with one set of lengths computes what the lengths hold when it runs."""
    x, qlens, kvlens, mode, layout = _inputs("heads_128")
    a = _call(x, mode=mode, **_buffers(x))
    b = _call(x, mode=mode, **_buffers(x))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        c = _call(x, mode=mode, **_buffers(x))
    torch.cuda.current_stream().wait_stream(s)
    for u, v, w in zip(a, b, c):
        assert torch.equal(u, v) and torch.equal(u, w)
    buf = _buffers(x)
    p = sfa.make_paged_params(x["cache"], x["block_table"], x["act_seq_kv"], tokens=x["q"].shape[0], heads=128,
                              layout="TND", act_seq_q=x["act_seq_q"])
    ws = torch.empty(sfa.paged_workspace_size(p), dtype=torch.uint8, device="cuda")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = _call(x, mode=mode, workspace=ws, **buf)
    x["act_seq_kv"].copy_(torch.tensor([900, 64, 17], dtype=torch.int32))
    x["act_seq_q"].copy_(torch.tensor([2, 1, 1], dtype=torch.int32))
    for _ in range(2):
        for t in got:
            t.fill_(UNTOUCHED)
        g.replay()
        torch.cuda.synchronize()
        _check(x, got, [2, 1, 1], [900, 64, 17])
    assert sfa.read_device_error(ws) == 0


@pytest.mark.gpu
@pytest.mark.parametrize("what", ["negative q", "negative kv", "q over T1", "kv over table"])
def test_paged_bad_lengths(what):
    x, qlens, kvlens, mode, layout = _inputs("heads_3")
    ws = torch.full((64 << 20,), 255, dtype=torch.uint8, device="cuda")
    key, val = {"negative q": ("act_seq_q", -1), "negative kv": ("act_seq_kv", -5), "q over T1": ("act_seq_q", 51),
                "kv over table": ("act_seq_kv", x["block_table"].shape[1] * 48 + 1)}[what]
    old = int(x[key][2])
    x[key][2] = val
    for t in _call(x, workspace=ws, **_buffers(x)):
        assert bool((t == UNTOUCHED).all())
    assert sfa.read_device_error(ws) == 2
    x[key][2] = old
    got = _call(x, workspace=ws, **_buffers(x))
    assert sfa.read_device_error(ws) == 0
    _check(x, got, qlens, kvlens)


@pytest.mark.gpu
@pytest.mark.parametrize("page", [-1, 1 << 30, 2 ** 31 - 1])
def test_paged_bad_page(page):
    """A table entry outside the cache is reported and disturbs only its sequence."""
    x, qlens, kvlens, mode, layout = _inputs("heads_3")
    ws = torch.empty(64 << 20, dtype=torch.uint8, device="cuda")
    want = _call(x, workspace=ws, **_buffers(x))[0]
    assert sfa.read_device_error(ws) == 0
    x["block_table"][1, 1] = page
    out = _call(x, workspace=ws, **_buffers(x))[0]
    assert sfa.read_device_error(ws) == 3
    assert torch.equal(out[:1], want[:1]) and torch.equal(out[8:], want[8:])


@pytest.mark.gpu
def test_paged_empty():
    x = paged_inputs([0, 0], [5, 0], 4, "bf16")
    ws = torch.full((64 << 20,), 255, dtype=torch.uint8, device="cuda")
    out, _, _ = _call(x, workspace=ws)
    assert out.shape == (0, 4, 512) and sfa.read_device_error(ws) == 0
    x = paged_inputs([0, 0], [5, 0], 4, "bf16", extra=3)
    for t in _call(x, workspace=ws, **_buffers(x)):
        assert bool((t == UNTOUCHED).all())
    assert sfa.read_device_error(ws) == 0


# ------------------------------------------------------------------ a serving run
@pytest.mark.gpu
@pytest.mark.parametrize("heads", [16, 128])
def test_prompt_then_steps(heads):
    """A prompt in two chunks and single-token steps through append and
    attention, against norm_rope and the framework's forward over contiguous
    rows with every earlier key selected."""
    torch.manual_seed(0)
    n, page, dt = 150, 32, DTYPES["bf16"]
    r = lambda *s: torch.randn(*s, device="cuda").to(dt)  # noqa: E731
    k, kr, q, qr, w, cs = r(n, 1, 512), r(n, 1, 64), r(n, heads, 512), r(n, heads, 64), r(512), table(n, "cuda")
    pos = torch.arange(n, dtype=torch.int32, device="cuda")
    _, qro, ko, kro, _, _ = sfa.norm_rope(pos, cs, k=k, k_weight=w, k_rope=kr, q_rope=qr)
    idx = torch.arange(n, dtype=torch.int32, device="cuda").repeat(n, 1)
    want, wmax, wsum = sfa.fwd(q[None], ko[None], ko[None], idx.view(1, n, 1, n), SCALE, q_rope=qro[None],
                               k_rope=kro[None], sparse_mode=3)
    cache = torch.full((8, page, 576), float("nan"), dtype=dt, device="cuda")
    bt = torch.tensor([[3, 0, 7, 1, 5]], dtype=torch.int32, device="cuda")
    done = 0
    for new in (70, 75, 1, 1, 1, 2):
        s = slice(done, done + new)
        done += new
        kv = torch.tensor([done], dtype=torch.int32, device="cuda")
        _, got_qr = sfa.cache_append(cache, bt, kv, k[None, s], kr[None, s], cs, k_weight=w, q_rope=qr[None, s])
        assert torch.equal(got_qr[0], qro[s])
        out, smax, ssum = sfa.paged_fwd(q[None, s], cache, bt, kv, SCALE, q_rope=got_qr)
        # both round P (the forward three times) and the result: at most four
        # half steps of values whose weighted mean of magnitudes is below 1.5 rms
        lim = 5 * 2.0 ** -8 * ko.float().abs().max()
        assert float((out[0].float() - want[0, s].float()).abs().max()) <= float(lim)
        # each side's score is off by at most 64 units of 2^-24 times
        # scale |q| |k| (the bound of latent_util.paged_bound; 576 products):
        # d apart by at most 2 d, and the sums of exponentials by 4 d
        d = 64 * U32 * SCALE * torch.cat((q[s], qro[s]), -1).float().norm(dim=-1) * \
            torch.cat((ko, kro), -1).float().norm(dim=-1).max()
        assert bool(((smax[0, 0] - wmax[0, 0, s]).abs() <= 2 * d + U32 * 8).all())
        assert bool(((ssum[0, 0] / wsum[0, 0, s] - 1).abs() <= 4 * d + 1e-4).all())
    assert done == n
