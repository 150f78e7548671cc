"""Attention over the paged cache for few query rows a sequence (row tiles of
32 or 64): calls whose sequences have at most 64 (token, head) rows on the mean and
whose block tables can hold a long cache."""
import pytest
import torch

import sfa_grad_gb300 as sfa
from latent_util import paged_inputs
from test_paged import SCALE, UNTOUCHED, _buffers, _call, _check

pytestmark = pytest.mark.gpu

CAPACITY = 200_000     # keys that the tables can hold in all, past the kernel's threshold


def _wide(x):
    """The same call with a block table for longer sequences (its further
    entries lie outside the cache)."""
    bt, page = x["block_table"], x["cache"].shape[1]
    width = max(bt.shape[1], -(-CAPACITY // (page * bt.shape[0])))
    out = torch.full((bt.shape[0], width), -5, dtype=torch.int32, device=bt.device)
    out[:, :bt.shape[1]] = bt
    return dict(x, block_table=out)


CASES = {
    # qlens, kvlens, heads, dtype, page, rope, mode, layout, s1, extra
    "one_key": ([1], [1], 1, "bf16", 16, True, 3, "BSND", 1, 0),
    "no_key": ([1, 2, 3], [0, 1, 0], 4, "fp16", 16, True, 3, "TND", None, 0),
    "borders": ([1] * 11, [1, 62, 63, 64, 65, 127, 128, 129, 255, 256, 257], 16, "bf16", 64, True, 3, "TND", None, 3),
    "heads_32": ([1] * 5, [700, 64, 1, 130, 2000], 32, "bf16", 128, True, 3, "BSND", 1, 0),
    "heads_17": ([1, 0, 1, 1], [400, 90, 33, 70], 17, "fp16", 48, True, 3, "TND", None, 2),
    "heads_33": ([1] * 6, [700, 64, 1, 130, 2000, 63], 33, "fp16", 128, True, 3, "BSND", 1, 0),
    "heads_64": ([1] * 5 + [0], [900, 65, 1, 128, 3000, 70], 64, "bf16", 64, True, 3, "TND", None, 1),
    "drafts_60": ([3, 2, 1, 0], [500, 2, 64, 67], 20, "bf16", 32, True, 3, "BSND", 3, 0),
    "no_mask_64": ([1, 2], [200, 40], 32, "fp16", 48, True, 0, "TND", None, 0),
    "no_rope_64": ([1, 1, 1], [500, 129, 3], 50, "bf16", 64, False, 3, "TND", None, 0),
    "long_64": ([1], [30000], 64, "bf16", 64, True, 3, "BSND", 1, 0),
    "uneven_64": ([40] + [1] * 30, [300] + list(range(1, 31)), 24, "fp16", 16, True, 3, "TND", None, 0),
    "drafts": ([3, 2, 1, 4], [500, 2, 64, 67], 8, "bf16", 32, True, 3, "BSND", 4, 0),
    "more_new_than_cached": ([4, 4], [3, 70], 5, "fp16", 16, True, 3, "BSND", 4, 0),
    # a few tokens on the mean, many of one sequence: several row tiles of it
    "uneven": ([60] + [1] * 40, [300] + list(range(1, 41)), 10, "bf16", 64, True, 3, "TND", None, 0),
    "no_mask": ([1, 2], [200, 40], 12, "bf16", 64, True, 0, "TND", None, 0),
    "no_rope": ([1, 2, 1], [500, 129, 3], 16, "bf16", 64, False, 3, "TND", None, 0),
    "large_page": ([1, 1], [1025, 1023], 9, "fp16", 1024, True, 3, "TND", None, 0),
    # pieces: one sequence over all SMs, of many and of few pieces
    "long": ([1], [30000], 16, "bf16", 64, True, 3, "BSND", 1, 0),
    "long_3": ([1, 2, 1], [9000, 20, 4000], 16, "fp16", 16, True, 3, "TND", None, 0),
    "many": ([1] * 200, [1 + (i * 37) % 300 for i in range(200)], 16, "bf16", 32, True, 3, "BSND", 1, 0),
}


def _inputs(name, **over):
    qlens, kvlens, heads, dtype, page, rope, mode, layout, s1, extra = CASES[name]
    x = paged_inputs(qlens, kvlens, heads, dtype, page=page, rope=rope, layout=layout, s1=s1, extra=extra, **over)
    return _wide(x), qlens, kvlens, mode, layout


@pytest.mark.parametrize("name", list(CASES))
def test_few(name):
    x, qlens, kvlens, mode, layout = _inputs(name)
    _check(x, _call(x, mode=mode, layout=layout, **_buffers(x)), qlens, kvlens, mode=mode, layout=layout)


@pytest.mark.parametrize("name", ["long_3", "heads_64"])
@pytest.mark.parametrize("scale", [0.7, -SCALE, 0.0])
def test_few_scales(scale, name):
    x, qlens, kvlens, mode, layout = _inputs(name)
    _check(x, _call(x, scale, mode, layout, **_buffers(x)), qlens, kvlens, scale, mode, layout)


@pytest.mark.parametrize("heads,dtype", [(16, "bf16"), (32, "fp16"), (64, "bf16")])
def test_few_rising_scores(heads, dtype):
    """Scores that rise along the keys, so that O is rescaled tile after tile."""
    qlens, kvlens = [1, 1], [2500, 90]
    x = _wide(paged_inputs(qlens, kvlens, heads, dtype, k_scale=0.3))
    for b, m in enumerate(kvlens):
        j = torch.arange(m, device="cuda")
        rows = x["block_table"][b][j // 64].long() * 64 + j % 64
        ramp = (torch.arange(m, device="cuda") / m * 0.9 + 0.1)[:, None]
        keys = x["q"][b, 0].float() * ramp
        x["cache"].flatten(0, 1)[rows, :512] = keys.to(x["cache"].dtype)
    _check(x, _call(x, 0.3, **_buffers(x)), qlens, kvlens, 0.3)


@pytest.mark.parametrize("heads", [16, 32])
def test_few_nan_ahead(heads):
    """Non-finite rows of the cache reach only the tokens that see them."""
    qlens, kvlens = [3, 1], [130, 70]
    x = _wide(paged_inputs(qlens, kvlens, heads, "bf16"))
    clean = _call(x, **_buffers(x))[0]
    flat = x["cache"].flatten(0, 1)
    for at, v in ((128, float("inf")), (129, float("nan"))):      # seen by tokens 1 and 2, and by token 2
        flat[x["block_table"][0, at // 64].long() * 64 + at % 64] = v
    out = _call(x, **_buffers(x))[0]
    assert torch.equal(out[0], clean[0]) and torch.equal(out[3], clean[3])
    assert bool(out[1].isnan().any()) and bool(out[2].isnan().any())


def test_few_same_bits_and_graph():
    x, qlens, kvlens, mode, layout = _inputs("many")
    a = _call(x, mode=mode, layout=layout, **_buffers(x))
    b = _call(x, mode=mode, layout=layout, **_buffers(x))
    assert all(torch.equal(u, v) for u, v in zip(a, b))
    buf, ws = _buffers(x), torch.empty(64 << 20, dtype=torch.uint8, device="cuda")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = _call(x, mode=mode, layout=layout, workspace=ws, **buf)
    kvlens = [max(1, k // 2) for k in kvlens]
    x["act_seq_kv"].copy_(torch.tensor(kvlens, dtype=torch.int32))
    for _ in range(2):
        for t in got:
            t.fill_(UNTOUCHED)
        g.replay()
        torch.cuda.synchronize()
        _check(x, got, qlens, kvlens, mode=mode, layout=layout)
    assert sfa.read_device_error(ws) == 0


@pytest.mark.parametrize("page", [-1, 1 << 30, 2 ** 31 - 1])
def test_few_bad_page(page):
    x, qlens, kvlens, mode, layout = _inputs("heads_17")
    ws = torch.empty(64 << 20, dtype=torch.uint8, device="cuda")
    want = _call(x, workspace=ws, **_buffers(x))[0]
    assert sfa.read_device_error(ws) == 0
    x["block_table"][0, 1] = page
    out = _call(x, workspace=ws, **_buffers(x))[0]
    assert sfa.read_device_error(ws) == 3
    assert torch.equal(out[1:], want[1:])


@pytest.mark.parametrize("what", ["negative q", "negative kv", "q over T1", "kv over table"])
def test_few_bad_lengths(what):
    x, qlens, kvlens, mode, layout = _inputs("heads_17")
    ws = torch.full((64 << 20,), 255, dtype=torch.uint8, device="cuda")
    key, val = {"negative q": ("act_seq_q", -1), "negative kv": ("act_seq_kv", -5), "q over T1": ("act_seq_q", 51),
                "kv over table": ("act_seq_kv", x["block_table"].shape[1] * 48 + 1)}[what]
    old = int(x[key][2])
    x[key][2] = val
    for t in _call(x, workspace=ws, **_buffers(x)):
        assert bool((t == UNTOUCHED).all())
    assert sfa.read_device_error(ws) == 2
    x[key][2] = old
    _check(x, _call(x, workspace=ws, **_buffers(x)), qlens, kvlens)
    assert sfa.read_device_error(ws) == 0


@pytest.mark.parametrize("name", ["long", "many", "long_64"])
def test_few_wait_timeout_then_recovery(name):
    """As the other kernels': a limit of a microsecond ends the call early or
    every wait was shorter, and the next call on the workspace is right."""
    x, qlens, kvlens, mode, layout = _inputs(name)
    ws = torch.empty(64 << 20, dtype=torch.uint8, device="cuda")
    got = _call(x, mode=mode, layout=layout, workspace=ws, wait_limit_us=1, **_buffers(x))
    code = sfa.read_device_error(ws)
    assert code in (0, 1)
    if code == 0:
        _check(x, got, qlens, kvlens, mode=mode, layout=layout)
    got = _call(x, mode=mode, layout=layout, workspace=ws, **_buffers(x))
    assert sfa.read_device_error(ws) == 0
    _check(x, got, qlens, kvlens, mode=mode, layout=layout)


@pytest.mark.parametrize("heads", [32, 64])
def test_few_and_many_rows_agree(heads):
    """The same sequences through both kernels (by the table's width): equal
    up to the two orders of summation."""
    kvlens = [500, 64, 65, 900, 1, 300]
    x = paged_inputs([1] * 6, kvlens, heads, "bf16")
    a = _call(x, **_buffers(x))
    b = _call(_wide(x), **_buffers(x))
    _check(x, a, [1] * 6, kvlens)
    _check(x, b, [1] * 6, kvlens)
    assert not all(torch.equal(u, v) for u, v in zip(a, b))     # two kernels indeed
