"""The position rotation with several axes (time, height, width), its
gradient, and the norm beside it."""
import ctypes

import pytest
import torch

import sfa_grad_gb300 as sfa
from latent_util import DTYPES, U32, floor_of, half_step, norm, table

EPS = 1e-6


def _turn(x, cs, pos, which, interleaved, back=False):
    """(tokens, heads, 64) in 64 bits; padding tokens give zeros."""
    x, cs = x.double(), cs.double()
    ok = ((pos >= 0) & (pos < cs.shape[0])).all(0)
    row = torch.where(ok, pos, 0).long()[which].T
    i = torch.arange(32, device=x.device)
    c, s = cs[row, i][:, None], cs[row, 32 + i][:, None] * (-1 if back else 1)
    a, b = (x[..., 0::2], x[..., 1::2]) if interleaved else (x[..., :32], x[..., 32:])
    u, v = a * c - b * s, b * c + a * s
    y = torch.stack((u, v), -1).flatten(-2) if interleaved else torch.cat((u, v), -1)
    return torch.where(ok[:, None, None], y, 0.0)


def _near(got, want, x, dt):
    # two products and a sum in fp32, one rounding to dtype
    tol = x.double().abs().amax(-1, keepdim=True) * 4 * U32 + want.abs() * half_step(dt) * 1.01 + floor_of(dt)
    assert bool(((got.double() - want).abs() <= tol).all())


SECTIONS = {"one": [0] * 32, "split": [0] * 8 + [1] * 12 + [2] * 12, "turns": [i % 3 for i in range(32)],
            "four": [3, 2, 1, 0] * 8, "last": [2] * 32, "first_unused": [1] * 16 + [2] * 16}


@pytest.mark.gpu
@pytest.mark.parametrize("sections", list(SECTIONS))
@pytest.mark.parametrize("interleaved", [True, False])
@pytest.mark.parametrize("tokens,heads,dtype", [(1, 1, "bf16"), (1, 128, "fp16"), (7, 33, "bf16"), (300, 16, "fp16"), (1025, 3, "bf16")])
def test_rotation_and_gradient(sections, interleaved, tokens, heads, dtype):
    t = DTYPES[dtype]
    g = torch.Generator().manual_seed(tokens)
    which = torch.tensor(SECTIONS[sections])
    n = int(which.max()) + 1 if sections != "one" else 3
    pos = torch.randint(0, 77, (n, tokens), generator=g)
    if tokens > 4:      # padding on any axis
        pos[0, 1], pos[n - 1, 2], pos[0, 3] = -1, 77, 2 ** 31 - 1
    cs = table(77)
    q, k = torch.randn(tokens, heads, 64, generator=g).to(t), torch.randn(tokens, 1, 64, generator=g).to(t)
    P = pos.int().cuda().contiguous()
    _, qo, _, ko, _, _ = sfa.norm_rope(P, cs.cuda(), k_rope=k.cuda(), q_rope=q.cuda(), interleaved=interleaved,
                                       axes=SECTIONS[sections])
    for x, y in ((q, qo), (k, ko)):
        _near(y.cpu(), _turn(x, cs, pos, which, interleaved), x, t)
    _, dq, _, dk, _, _ = sfa.norm_rope_grad(P, cs.cuda(), dk_rope=k.cuda(), dq_rope=q.cuda(), interleaved=interleaved,
                                            axes=tuple(SECTIONS[sections]))
    for x, y in ((q, dq), (k, dk)):
        _near(y.cpu(), _turn(x, cs, pos, which, interleaved, True), x, t)


@pytest.mark.gpu
def test_gradient_against_differences():
    """The gradient of a weighted sum of the outputs against its differences along random directions (the
    rotation is linear: a difference of two outputs is exact but for their rounding)."""
    g = torch.Generator().manual_seed(2)
    t, axes = torch.float16, SECTIONS["turns"]
    pos, cs = torch.randint(0, 50, (3, 20), generator=g).int().cuda(), table(50).cuda()
    x, d, w = (torch.randn(20, 5, 64, generator=g).to(t).cuda() for _ in range(3))
    f = lambda v: sfa.norm_rope(pos, cs, q_rope=v, axes=axes)[1].double()  # noqa: E731
    grad = sfa.norm_rope_grad(pos, cs, dq_rope=w, axes=axes)[1].double()
    up, down = (x + d), (x - d)
    step = (up.double() - down.double())
    lhs, rhs = ((f(up) - f(down)) * w.double()).sum(), (grad * step).sum()
    u = half_step(t)
    # each of the outputs and of the gradient's elements is one rounding off
    tol = u * ((f(up).abs() + f(down).abs()) * w.double().abs()).sum() + u * (grad.abs() * step.abs()).sum()
    assert abs(lhs - rhs) <= tol * 1.05
    # such roundings add up like a random walk; a wrong sign or pair is of the size of the sum's terms
    assert abs(lhs - rhs) <= 0.05 * ((grad * step).square().sum().sqrt())


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_norm_beside_it(dtype):
    """Keys normed and rotated in one call and their gradients; a token that is padding on one axis is zero
    in all rows and adds nothing to the weight's gradient."""
    t, u = DTYPES[dtype], half_step(DTYPES[dtype])
    g = torch.Generator().manual_seed(6)
    n, axes = 65, SECTIONS["split"]
    pos = torch.randint(0, 40, (3, n), generator=g)
    pos[2, 10], pos[1, 64] = 40, -3
    ok = torch.ones(n, dtype=torch.bool)
    ok[10] = ok[64] = False
    cs, P = table(40).cuda(), pos.int().cuda()
    k, kr, dy, dkr = (torch.randn(n, 1, w, generator=g).to(t).cuda() for w in (512, 64, 512, 64))
    wt = (1 + 0.1 * torch.randn(512, generator=g)).to(t).cuda()
    _, _, y, yr, _, rstd = sfa.norm_rope(P, cs, k=k, k_weight=wt, k_rope=kr, eps=EPS, axes=axes)
    want, r = norm(k.cpu(), wt.cpu(), EPS)
    want = torch.where(ok[:, None, None], want, 0.0)
    assert bool(((y.cpu().double() - want).abs() <= want.abs() * (u * 1.01 + 20 * U32)).all())
    assert not bool(y[10].any()) and not bool(yr[64].any()) and rstd[10].item() == 0
    _, _, dk, dkr2, _, dw = sfa.norm_rope_grad(P, cs, k=k, k_weight=wt, k_rstd=rstd, dk=dy, dk_rope=dkr, axes=axes)
    x = k.cpu().double().requires_grad_()
    w = wt.cpu().double().requires_grad_()
    out = x / (x.square().mean(-1, keepdim=True) + EPS).sqrt() * w
    (torch.where(ok[:, None, None], out, 0.0) * dy.cpu().double()).sum().backward()
    # sums of 512 products in fp32 and one rounding
    scale = x.grad.abs().amax(-1, keepdim=True)
    assert bool(((dk.cpu().double() - x.grad).abs() <= x.grad.abs() * u * 1.01 + scale * 64 * U32).all())
    terms = (dy.cpu().double() * x.detach() * r[..., None]).abs().sum((0, 1))
    assert bool(((dw.cpu().double() - w.grad).abs() <= terms * 64 * U32).all())
    _near(dkr2.cpu(), _turn(dkr.cpu(), cs.cpu(), pos, torch.tensor(axes), True, True), dkr.cpu(), t)


@pytest.mark.gpu
def test_equal_axes_are_one_axis():
    """The same position on every axis: the bits of the call with one; in place, and through a graph."""
    g = torch.Generator().manual_seed(8)
    pos = torch.randint(0, 60, (130,), generator=g).int().cuda()
    cs, q = table(60).cuda(), torch.randn(130, 17, 64, generator=g).bfloat16().cuda()
    one = sfa.norm_rope(pos, cs, q_rope=q)[1]
    many = pos.expand(4, -1).contiguous()
    assert torch.equal(sfa.norm_rope(many, cs, q_rope=q, axes=SECTIONS["four"])[1], one)
    assert torch.equal(sfa.norm_rope(pos[None].contiguous(), cs, q_rope=q, axes=SECTIONS["one"])[1], one)
    x = q.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        sfa.norm_rope(many, cs, q_rope=x, axes=SECTIONS["four"], outputs=(None, x, None, None, None, None))
    x.copy_(q)
    graph.replay()
    assert torch.equal(x, one)


def test_refusals():
    from sfa_grad_gb300.latent import RowsParams, _lib
    L, f = _lib(), ctypes.c_void_p(256)
    p = ctypes.byref(RowsParams(0, 1, 3, 4, 9, EPS))
    ok = bytes(32)
    for n, at, code in ((0, ok, sfa.SFA_ERR_PARAM_INVALID), (5, ok, sfa.SFA_ERR_PARAM_INVALID), (3, None, sfa.SFA_ERR_NULLPTR),
                        (2, bytes([2] + [0] * 31), sfa.SFA_ERR_PARAM_INVALID)):
        assert L.sfa_norm_rope_axes(p, n, at, *[f] * 15, None) == code
        assert L.sfa_norm_rope_axes_grad(p, n, at, *[f] * 19, 1 << 40, None) == code
    # several axes need their positions, whatever rows are there
    a = [f] * 15
    a[0] = None
    assert L.sfa_norm_rope_axes(p, 3, ok, *a, None) == sfa.SFA_ERR_NULLPTR
    cs, q = torch.zeros(9, 64), torch.zeros(5, 2, 64, dtype=torch.bfloat16)
    for shape, axes in (((5,), [0] * 32), ((3, 4), [0] * 32), ((5, 5), [0] * 32), ((3, 5), [3] * 32), ((3, 5), [0] * 31)):
        pos = torch.zeros(shape, dtype=torch.int32)
        with pytest.raises(ValueError, match="axes|positions"):
            sfa.norm_rope(pos, cs, q_rope=q, axes=axes)
        with pytest.raises(ValueError, match="axes|positions"):
            sfa.norm_rope_grad(pos, cs, dq_rope=q, axes=axes)
    with pytest.raises(ValueError, match="positions"):
        sfa.norm_rope(None, None, k=torch.zeros(5, 1, 512, dtype=torch.bfloat16), axes=[0] * 32,
                      k_weight=torch.zeros(512, dtype=torch.bfloat16))
