"""What positions cost rows that are normed and not turned."""
import pytest
import torch

import sfa_grad_gb300 as sfa
from latent_util import DTYPES
from timing_util import in_turns


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,interleaved", [("fp16", True), ("bf16", False)])
def test_positions_cost_normed_rows_nothing(dtype, interleaved):
    """They only say which tokens are padding.  The same rows with and without: the same results, and times
    that differ by the reads of them (a kernel that also held several axes' positions took 16 % more)."""
    t, n, heads = DTYPES[dtype], 8191, 16
    g = torch.Generator(device="cuda").manual_seed(1)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda").to(t)  # noqa: E731
    k, q, w = r(n, 1, 512), r(n, heads, 512), r(512)
    pos = torch.randint(0, 4096, (n,), generator=g, device="cuda").int()
    cs = torch.randn(4096, 64, generator=g, device="cuda")
    new = lambda: tuple(None if h is None else torch.empty(n, *h, dtype=d, device="cuda") for h, d in (  # noqa: E731
        ((heads, 512), t), (None, t), ((1, 512), t), (None, t), ((heads,), torch.float32), ((1,), torch.float32)))
    a, b = new(), new()
    kw = dict(k=k, k_weight=w, q=q, q_weight=w, interleaved=interleaved)
    with_, without = in_turns(lambda: sfa.norm_rope(pos, cs, outputs=a, **kw),
                              lambda: sfa.norm_rope(None, None, outputs=b, **kw))
    assert all(x is None or torch.equal(x, y) for x, y in zip(a, b))
    assert with_ <= 1.12 * without, (with_, without)
