"""The 4-bit cache at its edges: waits that run out, bad pages beside them,
offsets past 32 bits, the numbers of rows at which another kernel takes a
call, workspaces, random shapes."""
import random
import time

import pytest
import torch

import sfa_grad_gb300 as sfa
from cache4_util import packed_inputs, packed_rows, values
from latent_util import DTYPES, table
from test_cache4 import SCALE, _buffers, _call, _check

pytestmark = pytest.mark.gpu


def _workspace():
    return torch.empty(192 << 20, dtype=torch.uint8, device="cuda")


# ------------------------------------------------------------------ kernels
# Rows a sequence, on the mean: up to 32 single CTAs, up to 512 pairs, beyond
# unpacked ahead.
PATHS = {
    "32": ([1, 1], [700, 90], 32), "33": ([1, 1], [700, 90], 33), "512": ([4, 4], [700, 90], 128),
    "640": ([5, 5], [700, 90], 128), "32_of_many": ([8] + [0] * 7, [300] + [5] * 7, 32),
    "mean_of_uneven": ([40, 0, 0, 0, 0], [300, 1, 1, 1, 1], 64), "mean_beyond": ([90, 1], [300, 20], 128),
}


@pytest.mark.parametrize("name", list(PATHS))
@pytest.mark.parametrize("dtype,page,rope", [("bf16", 64, True), ("fp16", 48, False)])
def test_rows_a_sequence(name, dtype, page, rope):
    qlens, kvlens, heads = PATHS[name]
    x = packed_inputs(qlens, kvlens, heads, dtype, page=page, rope=rope)
    _check(x, _call(x, **_buffers(x, "TND")), qlens, kvlens)


@pytest.mark.parametrize("seed", range(24))
def test_random_calls(seed):
    r = random.Random(seed)
    batch = r.choice((1, 2, 5, 17))
    heads = r.choice((1, 3, 8, 16, 24, 40, 64, 100, 128))
    qlens = [r.choice((0, 1, 1, 1, 2, r.randint(1, 9))) for _ in range(batch)]
    kvlens = [max(0, r.choice((q, q + r.randint(0, 20), r.randint(0, 600), r.randint(0, 3000)))) for q in qlens]
    mode = r.choice((0, 3, 3))
    layout = r.choice(("TND", "BSND"))
    x = packed_inputs(qlens, kvlens, heads, r.choice(("bf16", "fp16")), page=r.choice((16, 32, 48, 64, 80, 128, 256)),
                      rope=r.random() < 0.8, layout=layout, s1=max(qlens + [1]) + r.choice((0, 2)), extra=r.choice((0, 3)),
                      seed=seed, cache_scale=2.0 ** r.randint(-3, 2))
    _check(x, _call(x, mode=mode, layout=layout, **_buffers(x, layout)), qlens, kvlens, mode=mode, layout=layout)


@pytest.mark.parametrize("qlen,heads,need", [(1, 16, False), (4, 128, False), (5, 128, True)])
def test_workspace_sizes(qlen, heads, need):
    """Calls that unpack ahead need room for the pages their tables name, or for the cache's; a workspace of
    that size does, a smaller one is refused."""
    x = packed_inputs([qlen] * 2, [300, 40], heads, "bf16", page=16)
    p = sfa.make_paged_params(x["cache"], x["block_table"], x["act_seq_kv"], tokens=2 * qlen, heads=heads, layout="TND",
                              act_seq_q=x["act_seq_q"], dtype=torch.bfloat16)
    base, size = sfa.paged_workspace_size(p), sfa.paged4_workspace_size(p)
    pages = min(x["block_table"].numel(), x["cache"].shape[0])
    rows = pages * 16 * 576 * 2 if need else 0
    assert base + rows <= size <= base + rows + (x["block_table"].numel() * 4 + 256 if need else 0)
    ws = torch.empty(size, dtype=torch.uint8, device="cuda")
    _check(x, _call(x, workspace=ws, **_buffers(x, "TND")), [qlen] * 2, [300, 40])
    with pytest.raises(sfa.SfaError):
        _call(x, workspace=ws[:size - 256])


@pytest.mark.parametrize("spare", [0, 40])
def test_pages_unpacked_by_table_or_by_page(spare):
    """A cache with fewer pages than the tables have entries, its pages shared, and one with more."""
    qlens, kvlens = [9, 9, 9], [300, 280, 260]
    x = packed_inputs(qlens, kvlens, 128, "bf16", page=64, poison=False, spare=spare)
    x["block_table"][1:, :4] = x["block_table"][0, :4]
    _check(x, _call(x, **_buffers(x, "TND")), qlens, kvlens)
    x["block_table"][1, 1] = -4
    ws = _workspace()
    got = _call(x, workspace=ws, **_buffers(x, "TND"))
    assert sfa.read_device_error(ws) == 3
    zero = dict(x, cache=torch.cat((x["cache"], torch.zeros_like(x["cache"][:1]))), block_table=x["block_table"].clone())
    zero["block_table"][1, 1] = x["cache"].shape[0]
    assert all(torch.equal(a, b) for a, b in zip(got, _call(zero, **_buffers(x, "TND"))))


# ------------------------------------------------------------------ waits that run out
# A limit of a microsecond on cold caches: the first key tile's scores need the
# table's entry, the rows' way into shared memory and their unpacking, several
# microseconds that some warp waits for.  The limit runs out in every call, and the
# next call on the workspace is right.
WAITS = {
    "pairs_pieces": ([1], [30000], 128), "pairs_whole": ([4] * 40, [300 + 9 * i for i in range(40)], 128),
    "pairs_one_tile": ([1] * 5, [9] * 5, 64), "few_pieces": ([1], [30000], 16),
    "few_whole": ([1] * 200, [1 + (i * 37) % 300 for i in range(200)], 16), "unpacked": ([60, 3], [2000, 700], 128),
}


@pytest.mark.parametrize("name", list(WAITS))
def test_short_limit_runs_out(name):
    qlens, kvlens, heads = WAITS[name]
    x = packed_inputs(qlens, kvlens, heads, "bf16")
    ws, cold = _workspace(), torch.empty(256 << 20, dtype=torch.uint8, device="cuda")
    _call(x, workspace=ws)      # the library is loaded
    codes = []
    for _ in range(4):
        cold.fill_(1)
        torch.cuda.synchronize()
        t0 = time.perf_counter()
        _call(x, workspace=ws, wait_limit_us=1)
        torch.cuda.synchronize()
        # the wind-down waits only for work already issued: far below its own 2 s limit
        assert time.perf_counter() - t0 < 1.0
        codes.append(sfa.read_device_error(ws))
    assert codes == [1] * 4
    got = _call(x, workspace=ws, **_buffers(x, "TND"))
    assert sfa.read_device_error(ws) == 0
    _check(x, got, qlens, kvlens)


@pytest.mark.parametrize("heads", [16, 128])
@pytest.mark.parametrize("kvlen", [40, 180_000])
def test_timeout_is_not_lost_to_a_bad_page(heads, kvlen):
    x = packed_inputs([1], [40], heads, "bf16", page=16)
    x["block_table"] = torch.full((1, 200_000 // 16), -1, dtype=torch.int32, device="cuda")
    x["act_seq_kv"].fill_(kvlen)
    ws, cold = _workspace(), torch.empty(256 << 20, dtype=torch.uint8, device="cuda")
    _call(x, workspace=ws)
    assert sfa.read_device_error(ws) == 3
    codes = []
    for _ in range(10):
        cold.fill_(1)
        _call(x, workspace=ws, wait_limit_us=1)
        codes.append(sfa.read_device_error(ws))
    assert codes == [1] * 10


# ------------------------------------------------------------------ offsets past 32 bits
@pytest.mark.parametrize("heads,tokens", [(16, 1), (128, 1), (128, 7)])
def test_pages_past_32_bits(heads, tokens):
    """A cache of 4.9e9 bytes (2^32 is 4.3e9): its last pages are appended to, read and unpacked as a small
    cache's are, to the bit."""
    torch.manual_seed(0)
    page, far, t, n = 64, 184_000, DTYPES["bf16"], 150
    small = torch.zeros(4, page, 416, dtype=torch.uint8, device="cuda")
    big = torch.empty(far + 4, page, 416, dtype=torch.uint8, device="cuda")
    big[far:] = 0
    bt = torch.tensor([[2, 0, 3]], dtype=torch.int32, device="cuda")
    kv = torch.tensor([n], dtype=torch.int32, device="cuda")
    k, kr = torch.randn(1, n, 1, 512, device="cuda").to(t), torch.randn(1, n, 1, 64, device="cuda").to(t)
    q, qr = (torch.randn(1, tokens, heads, w, device="cuda").to(t) for w in (512, 64))
    cs, got = table(n, "cuda"), []
    for cache, b in ((small, bt), (big, bt + far)):
        sfa.cache_append(cache, b, kv, k, kr, cs, k_weight=k[0, 0, 0].contiguous())
        got.append(sfa.paged_fwd(q, cache, b, kv, SCALE, q_rope=qr))
    assert torch.equal(small, big[far:])
    assert bool(got[0][0].isfinite().all()) and bool((got[0][0] != 0).any())
    for a, b in zip(*got):
        assert torch.equal(a, b)
    slot = torch.tensor([(far + 1) * page + 5], dtype=torch.int32, device="cuda")
    sfa.cache_append_slots(big, slot, kv * 0 + 7, k[0, :1], kr[0, :1], cs)
    sfa.cache_append_slots(small, slot - far * page, kv * 0 + 7, k[0, :1], kr[0, :1], cs)
    assert torch.equal(small, big[far:])
    if heads == 16:
        out = torch.empty(far + 4, page, 576, dtype=t, device="cuda")
        sfa.cache_unpack(big, t, out=out)
        assert torch.equal(out[far:], sfa.cache_unpack(small, t))


# ------------------------------------------------------------------ streams
def test_calls_on_another_stream_and_in_place():
    """Append, values and attention on a stream of the caller's, q_rope turned in place."""
    t = DTYPES["fp16"]
    g = torch.Generator().manual_seed(0)
    cache = torch.zeros(8, 16, 416, dtype=torch.uint8, device="cuda")
    n = 40
    k, kr = torch.randn(n, 1, 512, generator=g).to(t).cuda(), torch.randn(n, 1, 64, generator=g).to(t).cuda()
    qr = torch.randn(n, 5, 64, generator=g).to(t).cuda()
    slots, cs = torch.arange(n, dtype=torch.int32, device="cuda"), table(n).cuda()
    want, turned = sfa.cache_append_slots(cache.clone(), slots, slots, k, kr, cs, q_rope=qr)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    own = qr.clone()
    s.wait_stream(torch.cuda.current_stream())
    got, out = sfa.cache_append_slots(cache, slots, slots, k, kr, cs, q_rope=own, q_rope_out=own, stream=s)
    dense = sfa.cache_unpack(got, t, stream=s)
    s.synchronize()
    assert out is own and torch.equal(own, turned) and torch.equal(got, want)
    assert torch.equal(dense.cpu().double(), values(want, t, 1.0))


def test_rows_of_any_bytes():
    """Codes and scales of any bytes (negative scales too) are read as they stand, by the attention as by the
    values."""
    g = torch.Generator().manual_seed(1)
    for heads in (16, 128):
        x = packed_inputs([1, 1], [200, 70], heads, "bf16")
        rows = packed_rows(x["cache"].shape[0] * 64, "bf16", g, True, 1.0, 3.0)
        rows[:, 256:288] |= (torch.randint(0, 2, rows[:, 256:288].shape, generator=g) * 128).to(torch.uint8)
        x["cache"] = rows.view(-1, 64, 416).cuda()
        x["dense"] = sfa.cache_unpack(x["cache"], torch.bfloat16)
        assert torch.equal(x["dense"].cpu().double(), values(x["cache"], torch.bfloat16, 1.0))
        _check(x, _call(x, **_buffers(x, "TND")), [1, 1], [200, 70])
