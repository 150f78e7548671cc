"""Scales and epsilons at the ends of their ranges."""
import ctypes

import pytest
import torch

import sfa_grad_gb300 as sfa
from latent_util import paged_inputs
from sfa_grad_gb300.latent import PagedParams, RowsParams, _lib
from test_paged import _buffers, _call, _check
from test_paged_few import _wide


def test_values_beyond_fp32_are_refused():
    """The kernels hold the scale, its product with log2(e) and eps in fp32; a
    value that is infinite there is refused."""
    n = ctypes.c_size_t(0)
    paged = lambda scale: _lib().sfa_paged_workspace_size(ctypes.byref(PagedParams(  # noqa: E731
        1, 0, 2, 0, 4, 16, 512, 64, 8, 64, 4, scale, 3, 1, 0)), ctypes.byref(n))
    rows = lambda eps: _lib().sfa_norm_rope_grad_workspace_size(ctypes.byref(RowsParams(0, 1, 3, 4, 9, eps)),  # noqa: E731
                                                                ctypes.byref(n))
    for scale in (0.0, -0.0, 1e-45, 1e-300, 2.3e38, -2.3e38):
        assert paged(scale) == 0, scale
    for scale in (2.4e38, -3.4e38, 1e39, -1e300, float("inf"), float("nan")):
        assert paged(scale) == sfa.SFA_ERR_SHAPE, scale
    for eps in (0.0, 1e-300, 3.4e38):
        assert rows(eps) == 0, eps
    for eps in (3.5e38, 1e300, -1e-6, float("inf"), float("nan")):
        assert rows(eps) == sfa.SFA_ERR_SHAPE, eps
    f = ctypes.c_void_p(256)
    p = PagedParams(1, 0, 2, 0, 3, 4, 512, 64, 8, 64, 2, 1.0, 3, 1, 0)
    args = [f, f, f, f, f, f, f, 1e300, f, 9, None, None, None, None]
    assert _lib().sfa_cache_append(ctypes.byref(p), *args) == sfa.SFA_ERR_SHAPE


@pytest.mark.gpu
@pytest.mark.parametrize("few,heads", [(False, 128), (True, 16)])
@pytest.mark.parametrize("size,scale", [(1e15, 0.0), (1e15, -0.0), (1e16, 1e-32 / 24), (1e17, -1e-34 / 24), (1e-16, 1e32 / 24)])
def test_rows_far_from_one(few, heads, size, scale):
    """Elements far from one with the scale that fits them, and with none: a
    scale of zero weighs every key alike, whatever its score."""
    qlens, kvlens = [1, 2], [300, 65]
    x = paged_inputs(qlens, kvlens, heads, "bf16", q_scale=size, k_scale=size)
    if few:
        x = _wide(x)
    _check(x, _call(x, scale, **_buffers(x)), qlens, kvlens, scale)
