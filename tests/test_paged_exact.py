"""Scores that fp32 holds exactly come out exactly: whole numbers, in any
order of summation."""
import pytest
import torch

import sfa_grad_gb300 as sfa  # noqa: F401
from latent_util import U32, paged_inputs
from test_paged import _buffers, _call
from test_paged_few import _wide

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("few,heads", [(False, 16), (False, 128), (True, 16), (True, 32), (True, 64)])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("rope", [True, False])
@pytest.mark.parametrize("scale", [2.0 ** -6, 576 ** -0.5, -0.3])
def test_whole_scores_are_exact(few, heads, dtype, rope, scale):
    """Elements are whole numbers of at most 8: every product is at most 64 and
    every partial sum a whole number below 2^16, whatever the order.  So the
    largest score is known to the bit, and softmax_max is its product with the
    scale, both in fp32."""
    kvlens = [700, 65, 1]
    x = paged_inputs([1, 1, 1], kvlens, heads, dtype, rope=rope)
    g = torch.Generator().manual_seed(3)
    for name in ("q", "q_rope", "cache"):
        if x[name] is not None:
            whole = torch.randint(-8, 9, x[name].shape, generator=g).to(x[name].dtype).cuda()
            x[name] = torch.where(x[name].isnan(), x[name], whole)
    if few:
        x = _wide(x)
    _, smax, ssum = _call(x, scale, **_buffers(x))
    flat = x["cache"].flatten(0, 1).double()
    for b, m in enumerate(kvlens):
        j = torch.arange(m, device="cuda")
        keys = flat[x["block_table"][b, j // 64].long() * 64 + j % 64]
        q = x["q"][b].double()
        if rope:
            q = torch.cat((q, x["q_rope"][b].double()), -1)
        s = q @ keys.T
        top = s.amax(-1) if scale > 0 else s.amin(-1)
        assert torch.equal(smax[0, b], top.float() * torch.tensor(scale, dtype=torch.float32, device="cuda"))
        # An exponent's error: the factor scale log2(e) is rounded three times
        # (scale, log2(e), their product), the reference's product and the
        # difference once each: at most 3 |x - top| + 2 |top| + |x - top| units
        # of 2^-24, and the exponential 2^-22 of itself.
        z = (s - top[:, None]) * scale
        reach = (4 * z.abs() + 2 * (top * scale).abs()[:, None]) * U32
        bound = (z.exp() * (1.1 * reach + 4 * U32)).sum(-1) + (64 + m / 16) * U32 * z.exp().sum(-1)
        assert bool(((ssum[0, b].double() - z.exp().sum(-1)).abs() <= bound).all())
