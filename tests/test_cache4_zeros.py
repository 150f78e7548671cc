"""Bytes of a 4-bit row, the signs of its zeros among them."""
import pytest
import torch

import sfa_grad_gb300 as sfa
from cache4_util import CODES, quantise
from latent_util import DTYPES, norm

EPS = 1e-6


def _bytes(y):
    """The rows' 288 bytes by the definition; a code has the sign of its element, zeros too."""
    mag, scales, bad = quantise(y)
    sign = torch.where(bad.repeat_interleave(16, -1), False, y.signbit())
    c = mag + 8 * sign
    return torch.cat((c[..., 0::2] + 16 * c[..., 1::2], scales), -1).to(torch.uint8)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("form", ["norm", "large weights", "plain"])
def test_bytes_do_not_depend_on_the_way(form, dtype):
    """Zeros of both signs, and small values that round to zero, in rows that fp32 decides, in rows near a
    border, in rows of 64 bits, with weights of both signs and zeros among them."""
    t, n = DTYPES[dtype], 4096
    g = torch.Generator().manual_seed(12)
    k = torch.randn(n, 512, generator=g)
    k[torch.rand(n, 512, generator=g) < 0.1] = 0.0
    k = torch.where(torch.rand(n, 512, generator=g) < 0.1, -0.0, k).to(t)
    k[5] = 0.0
    k[6] = -0.0
    k[7, :32] = -0.0
    w = None
    if form != "plain":
        w = torch.randn(512, generator=g)
        w[::37] = 0.0
        w[1::37] = -0.0
        if form == "large weights":
            w[40:48] = 2.0 ** 62 if dtype == "bf16" else 60000.0
        w = w.to(t)
    cache = torch.zeros(n // 16, 16, 288, dtype=torch.uint8, device="cuda")
    sfa.cache_append_slots(cache, torch.arange(n, dtype=torch.int32, device="cuda"), None, k[:, None].cuda(),
                           k_weight=None if w is None else w.cuda(), eps=EPS)
    y = k.double() if w is None else norm(k, w, EPS)[0]
    got, want = cache.view(n, 288).cpu(), _bytes(y)
    assert torch.equal(got[:, CODES:], want[:, CODES:])
    assert torch.equal(got[:, :CODES], want[:, :CODES])


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_signed_zeros_read_back(dtype):
    """A negative zero is a zero with its sign, in either type."""
    t = DTYPES[dtype]
    k = torch.zeros(16, 1, 512, dtype=t)
    k[:, 0, ::2] = -0.0
    k[8:, 0, 5] = 1.0
    cache = torch.zeros(1, 16, 288, dtype=torch.uint8, device="cuda")
    sfa.cache_append_slots(cache, torch.arange(16, dtype=torch.int32, device="cuda"), None, k.cuda())
    x = sfa.cache_unpack(cache, t).cpu()[0]
    want = k[:, 0].clone()
    want[8:, 5] = 66 / 64       # a sixth of 1 lies between scales of 10/64 and 11/64, nearer to the latter; its code is 6
    assert torch.equal(x, want) and torch.equal(x.signbit(), want.signbit())
