"""What the attention over a paged cache reports: table entries outside the
cache, waits that run out, and both in one call."""
import time

import pytest
import torch

import sfa_grad_gb300 as sfa
from latent_util import paged_inputs
from test_paged import _buffers, _call, _check
from test_paged_few import _wide

pytestmark = pytest.mark.gpu


def _workspace():
    return torch.empty(64 << 20, dtype=torch.uint8, device="cuda")


# ------------------------------------------------------------------ pages
# Every value an entry can have that is not a page, those that a kernel might
# use as marks of its own among them.
@pytest.mark.parametrize("few", [False, True])
@pytest.mark.parametrize("page", [-1, -2, -3, -2 ** 31, "num_pages", 2 ** 31 - 1])
def test_bad_page_is_reported_and_reads_as_zeros(few, page):
    qlens, kvlens, heads = [1, 0, 1, 1], [400, 90, 33, 70], 17
    x = paged_inputs(qlens, kvlens, heads, "fp16", page=48)
    if few:
        x = _wide(x)
    ws = _workspace()
    want = _call(x, workspace=ws, **_buffers(x))[0]
    assert sfa.read_device_error(ws) == 0
    # the same call over a page of zeros in the entry's place
    zero = dict(x, cache=torch.cat((x["cache"], torch.zeros_like(x["cache"][:1]))), block_table=x["block_table"].clone())
    zero["block_table"][0, 1] = x["cache"].shape[0]
    zeros = _call(zero, **_buffers(x))
    x["block_table"][0, 1] = x["cache"].shape[0] if page == "num_pages" else page
    got = _call(x, workspace=ws, **_buffers(x))
    assert sfa.read_device_error(ws) == 3
    assert all(torch.equal(a, b) for a, b in zip(got, zeros))
    assert torch.equal(got[0][1:], want[1:])


# ------------------------------------------------------------------ waits that run out
# A limit of a microsecond on cold caches.  The first key tile's scores need
# the table's entry, the rows' way into shared memory and 32 MMAs at least,
# each after the other: several microseconds, which some warp waits for.  So
# the limit runs out in every call, and the next call on the workspace is right.
WAITS = {
    # qlens, kvlens, heads, few
    "whole_tiles": ([60, 3], [2000, 700], 128, False),
    "pieces": ([1], [30000], 128, False),
    "one_tile": ([9] * 5, [9] * 5, 64, False),
    "few_pieces": ([1], [30000], 16, True),
    "few_whole": ([1] * 200, [1 + (i * 37) % 300 for i in range(200)], 16, True),
    "few_64": ([1], [30000], 64, True),
}


@pytest.mark.parametrize("name", list(WAITS))
def test_short_limit_runs_out(name):
    qlens, kvlens, heads, few = WAITS[name]
    x = paged_inputs(qlens, kvlens, heads, "bf16")
    if few:
        x = _wide(x)
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
    got = _call(x, workspace=ws, **_buffers(x))
    assert sfa.read_device_error(ws) == 0
    _check(x, got, qlens, kvlens)


# ------------------------------------------------------------------ both
@pytest.mark.parametrize("few", [False, True])
@pytest.mark.parametrize("kvlen", [40, 180_000])
def test_timeout_is_not_lost_to_a_bad_page(few, kvlen):
    """A call that gave up says so, whatever pages it meets before and after:
    its outputs are not complete.  One worker's single key tile, and many for
    every worker, all of whose pages are bad."""
    x = paged_inputs([1], [40], 16 if few else 128, "bf16", page=16)
    x["block_table"] = torch.full((1, 200_000 // 16), -1, dtype=torch.int32, device="cuda")
    x["act_seq_kv"].fill_(kvlen)
    ws, cold = _workspace(), torch.empty(256 << 20, dtype=torch.uint8, device="cuda")
    _call(x, workspace=ws)
    assert sfa.read_device_error(ws) == 3
    codes = []
    for _ in range(20):
        cold.fill_(1)
        _call(x, workspace=ws, wait_limit_us=1)
        codes.append(sfa.read_device_error(ws))
    assert codes == [1] * 20
