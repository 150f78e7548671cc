"""What the attention over a paged cache reports: table entries outside the
cache, waits that run out, and both in one call."""
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
