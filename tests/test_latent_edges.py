"""Calls of the latent-row operators at their edges: waits that run out,
offsets past 32 bits, other streams, graphs that are replayed after their
inputs changed, pointers that are not aligned."""
import ctypes
import time

import pytest
import torch

import sfa_grad_gb300 as sfa
from latent_util import DTYPES, paged_inputs, paged_ref, table

SCALE = 576 ** -0.5
EPS = 1e-6


def _call(x, **kw):
    return sfa.paged_fwd(x["q"], x["cache"], x["block_table"], x["act_seq_kv"], SCALE, q_rope=x["q_rope"],
                         layout="TND", act_seq_q=x["act_seq_q"], **kw)


def _rows(t, heads, *shape):
    return torch.randn(*shape, device="cuda").to(DTYPES[t])


def _right(x, got, qlens, kvlens):
    out = got[0]
    for rows, o, _, _, (bound, _, _) in paged_ref(x, qlens, kvlens, SCALE, 3):
        assert bool(((out[rows].double() - o).abs() <= bound).all())


def test_words_of_index_arrays_are_aligned():
    """int32 and fp32 arrays off a 4-byte boundary are refused by the C entries."""
    from sfa_grad_gb300.latent import PagedParams, RowsParams, _lib
    f, odd = ctypes.c_void_p(256), ctypes.c_void_p(258)
    p = PagedParams(1, 0, 2, 0, 3, 4, 512, 64, 8, 64, 2, SCALE, 3, 1, 0)
    for i in (3, 4, 5, 7, 8):                  # block table, lengths, softmax_max, softmax_sum
        a = [f] * 10
        a[i] = odd
        assert _lib().sfa_paged_fwd(ctypes.byref(p), *a, 1 << 40, None) == sfa.SFA_ERR_PARAM_INVALID, i
    for i in (1, 2, 3, 12):                    # block table, lengths, error
        a = [f, f, f, f, f, f, None, EPS, f, 9, None, None, None, None]
        a[i] = odd
        assert _lib().sfa_cache_append(ctypes.byref(p), *a) == sfa.SFA_ERR_PARAM_INVALID, i
    r = RowsParams(0, 1, 3, 4, 9, EPS)
    for i in (0, 12, 13):                      # positions, rstd
        a = [f] * 15
        a[i] = odd
        assert _lib().sfa_norm_rope(ctypes.byref(r), *a[:14], None) == sfa.SFA_ERR_PARAM_INVALID, i
    for i in (0, 4, 7, 16, 17):                # positions, rstd, gradients of the weights
        a = [f] * 19
        a[i] = odd
        assert _lib().sfa_norm_rope_grad(ctypes.byref(r), *a, 1 << 40, None) == sfa.SFA_ERR_PARAM_INVALID, i


# ------------------------------------------------------------------ waits that run out
# A wait limit of a microsecond: whole row tiles over many key tiles, pieces
# of one row tile (few rows over a long cache), masked values that the loading
# warps clean.  A wait first lets the hardware suspend the warp, for up to ten
# microseconds, and looks at the limit only after that: a call all of whose
# waits are shorter succeeds.  So each call here gives up (as most do, the
# first ones on cold caches above all) or is right, and the workspace is as
# good as new for the next one.
@pytest.mark.gpu
@pytest.mark.parametrize("qlens,kvlens,heads", [([60, 3], [2000, 700], 128), ([1], [30000], 128), ([9] * 5, [9] * 5, 64)])
def test_wait_timeout_then_recovery(qlens, kvlens, heads):
    x = paged_inputs(qlens, kvlens, heads, "bf16")
    ws = torch.empty(64 << 20, dtype=torch.uint8, device="cuda")
    cold = torch.empty(256 << 20, dtype=torch.uint8, device="cuda")
    _call(x, workspace=ws)      # the library is loaded
    for _ in range(4):
        cold.fill_(1)
        torch.cuda.synchronize()
        t0 = time.perf_counter()
        got = _call(x, workspace=ws, wait_limit_us=1)
        torch.cuda.synchronize()
        took = time.perf_counter() - t0
        # the wind-down waits only for work already issued: far below its own 2 s limit
        assert took < 1.0, f"timed-out call took {took:.2f} s"
        code = sfa.read_device_error(ws)
        assert code in (0, 1)
        if code == 0:
            _right(x, got, qlens, kvlens)
    got = _call(x, workspace=ws)
    assert sfa.read_device_error(ws) == 0
    _right(x, got, qlens, kvlens)


# ------------------------------------------------------------------ offsets past 32 bits
@pytest.mark.gpu
def test_pages_past_32_bits():
    """A cache of 4.9e9 elements (2^32 is 4.3e9): its last pages are appended
    to and read as a small cache's are, to the bit."""
    torch.manual_seed(0)
    page, far, heads, t = 64, 132_000, 16, DTYPES["bf16"]
    small = torch.zeros(4, page, 576, dtype=t, device="cuda")
    big = torch.empty(far + 4, page, 576, dtype=t, device="cuda")
    bt = torch.tensor([[2, 0, 3]], dtype=torch.int32, device="cuda")
    kv = torch.tensor([150], dtype=torch.int32, device="cuda")
    k, kr = _rows("bf16", 1, 1, 150, 1, 512), _rows("bf16", 1, 1, 150, 1, 64)
    q, qr, cs = _rows("bf16", 1, 1, 150, heads, 512), _rows("bf16", 1, 1, 150, heads, 64), table(150, "cuda")
    got = []
    for cache, b in ((small, bt), (big, bt + far)):
        _, qro = sfa.cache_append(cache, b, kv, k, kr, cs, k_weight=k[0, 0, 0].contiguous(), q_rope=qr)
        got.append(sfa.paged_fwd(q, cache, b, kv, SCALE, q_rope=qro))
    at = [(n // page, n % page) for n in range(150)]
    for n in (0, 63, 64, 149):
        pg, i = at[n]
        assert torch.equal(small[int(bt[0, pg]), i], big[far + int(bt[0, pg]), i])
    assert bool(got[0][0].isfinite().all()) and bool((got[0][0] != 0).any())
    for a, b in zip(*got):
        assert torch.equal(a, b)


@pytest.mark.gpu
def test_rows_past_32_bits():
    """33,000 tokens of 128 heads, 2.16e9 elements (2^31 is 2.15e9): the last
    tokens get what a call on them alone gives, to the bit."""
    torch.manual_seed(0)
    n, heads, tail, t = 33_000, 128, 40, DTYPES["fp16"]
    q = torch.randn(n, heads, 512, device="cuda", dtype=t)
    qr = torch.randn(n, heads, 64, device="cuda", dtype=t)
    w, cs = torch.randn(512, device="cuda", dtype=t), table(n, "cuda")
    pos = torch.arange(n, dtype=torch.int32, device="cuda")
    last = slice(n - tail, n)
    a = sfa.norm_rope(pos, cs, q=q, q_weight=w, q_rope=qr)
    b = sfa.norm_rope(pos[last].contiguous(), cs, q=q[last], q_weight=w, q_rope=qr[last])
    for i in (0, 1, 4):
        assert torch.equal(a[i][last], b[i])
    ga = sfa.norm_rope_grad(pos, cs, q=q, q_weight=w, q_rstd=a[4], dq=a[0], dq_rope=a[1])
    gb = sfa.norm_rope_grad(pos[last].contiguous(), cs, q=q[last], q_weight=w, q_rstd=b[4], dq=b[0], dq_rope=b[1])
    for i in (0, 1):
        assert torch.equal(ga[i][last], gb[i])
    del ga, gb, a, b
    # a sequence a token, all of them over the same few keys: a row tile each,
    # so no row is cut into pieces
    page = torch.randn(2, 64, 576, device="cuda", dtype=t)
    one = lambda m, v: torch.full((m,), v, dtype=torch.int32, device="cuda")  # noqa: E731
    run = lambda s, m: sfa.paged_fwd(q[s], page, torch.ones(m, 1, dtype=torch.int32, device="cuda"), one(m, 50),  # noqa: E731
                                     SCALE, q_rope=qr[s], layout="TND", act_seq_q=one(m, 1))
    for a, b in zip(run(slice(0, n), n), run(last, tail)):
        a = a[0] if a.dim() == 3 and a.shape[0] == 1 else a
        b = b[0] if b.dim() == 3 and b.shape[0] == 1 else b
        assert torch.equal(a[last], b)


# ------------------------------------------------------------------ streams, graphs
@pytest.mark.gpu
def test_memory_of_a_call_belongs_to_its_stream():
    """A call on another stream that is still to run keeps its workspace and
    outputs, whatever the current stream allocates meanwhile."""
    qlens, kvlens = [1, 1], [5000, 900]
    x = paged_inputs(qlens, kvlens, 32, "bf16")
    _right(x, _call(x), qlens, kvlens)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        torch.cuda._sleep(40_000_000)
    got = _call(x, stream=s)
    spoil = [torch.full((64 << 20,), 255, dtype=torch.uint8, device="cuda") for _ in range(3)]
    s.synchronize()
    _right(x, got, qlens, kvlens)
    del spoil


@pytest.mark.gpu
def test_two_streams_at_once():
    """Two calls that may run at the same time, each with its own workspace."""
    xs = [paged_inputs([40, 1], [900, 3000], 64, "bf16", seed=s) for s in (1, 2)]
    want = [_call(x) for x in xs]
    streams = [torch.cuda.Stream() for _ in xs]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(4):
        for i, s in enumerate(streams):
            got[i].append(_call(xs[i], stream=s))
    torch.cuda.synchronize()
    for i in range(2):
        for g in got[i]:
            assert all(torch.equal(a, b) for a, b in zip(g, want[i]))


@pytest.mark.gpu
def test_step_replayed_over_growing_lengths():
    """One decoding step (append and attention) captured once and replayed
    with the lengths, rows and queries of every next token."""
    torch.manual_seed(0)
    B, heads, page, t, lens = 3, 16, 16, DTYPES["bf16"], [15, 31, 100]
    bt = torch.randperm(B * 8).view(B, 8).int().cuda()
    cs = table(128, "cuda")
    kv = torch.tensor(lens, dtype=torch.int32, device="cuda")
    caches = [torch.randn(B * 8, page, 576, device="cuda").to(t)]
    caches.append(caches[0].clone())
    k, kr = _rows("bf16", 1, B, 1, 1, 512), _rows("bf16", 1, B, 1, 1, 64)
    q, qr, w = _rows("bf16", 1, B, 1, heads, 512), _rows("bf16", 1, B, 1, heads, 64), _rows("bf16", 1, 512)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")

    def step(cache):
        _, qro = sfa.cache_append(cache, bt, kv, k, kr, cs, k_weight=w, q_rope=qr, error=err)
        return sfa.paged_fwd(q, cache, bt, kv, SCALE, q_rope=qro)

    step(caches[0].clone())
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = step(caches[0])
    for _ in range(20):
        kv += 1
        for x in (k, kr, q, qr):
            x.copy_(torch.randn_like(x))
        g.replay()
        for a, b in zip(got, step(caches[1])):
            assert torch.equal(a, b)
    assert torch.equal(caches[0], caches[1]) and int(err) == 0


@pytest.mark.gpu
def test_append_of_more_tokens_than_there_are():
    """TND lengths that add up to more tokens than k has: the sequences that
    fit are written, the others are left out and reported."""
    cache = torch.full((4, 16, 576), 3.0, dtype=DTYPES["bf16"], device="cuda")
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    bt, err = i32(0, 1, 2, 3).view(2, 2), i32(0)
    k, kr = _rows("bf16", 1, 5, 1, 512), _rows("bf16", 1, 5, 1, 64)
    sfa.cache_append(cache, bt, i32(2, 9), k, kr, table(32, "cuda"), layout="TND", act_seq_q=i32(2, 4), error=err)
    assert int(err) == 2
    assert torch.equal(cache[0, :2, :512], k[:2, 0]) and bool((cache[0, 2:] == 3).all()) and bool((cache[1:] == 3).all())
