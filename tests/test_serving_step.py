"""A few steps of serving as a program runs them: the plan of a step, the
append by its slots with positions of three axes, the attention over the
cache, for rows of 4 and of 16 bits, against histories kept in 64 bits."""
import math

import pytest
import torch

import sfa_grad_gb300 as sfa
from cache4_util import MAGNITUDES, e4m3_values, quantise
from latent_util import DTYPES, U32, floor_of, half_step, norm, table

EPS, SCALE = 1e-6, 576 ** -0.5
AXES = [0] * 8 + [1] * 12 + [2] * 12


def _held(y, unit):
    codes, scales, _ = quantise(y / unit)
    v = torch.tensor(MAGNITUDES, dtype=torch.float64)[codes] * torch.where(y < 0, -1.0, 1.0)
    return (v.unflatten(-1, (32, 16)) * e4m3_values()[scales][..., None] * unit).flatten(-2)


def _turn(x, cs, pos):
    row, i = pos[torch.tensor(AXES)].T, torch.arange(32)
    c, s = cs.double()[row, i][:, None], cs.double()[row, 32 + i][:, None]
    a, b = x.double()[..., 0::2], x.double()[..., 1::2]
    return torch.stack((a * c - b * s, b * c + a * s), -1).flatten(-2)


@pytest.mark.gpu
@pytest.mark.parametrize("captured", [False, True])
@pytest.mark.parametrize("bits,dtype,heads", [(4, "bf16", 16), (4, "fp16", 128), (4, "bf16", 40), (16, "bf16", 16)])
def test_steps(bits, dtype, heads, captured):
    t, unit = DTYPES[dtype], 0.25 if bits == 4 else None
    u = half_step(t)
    batch, page, per, tokens = 6, 16, 20, 256
    g = torch.Generator().manual_seed(heads)
    dev = lambda x: x.cuda()  # noqa: E731
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32, device="cuda")  # noqa: E731
    pages = batch * per
    cache = torch.full((pages, page, 416), 255, dtype=torch.uint8, device="cuda") if bits == 4 else \
        torch.full((pages, page, 576), float("nan"), dtype=t, device="cuda")
    bt, kv, new, count = i32(batch, per), i32(batch), i32(batch), i32(1)
    count.fill_(pages)
    free = torch.randperm(pages, generator=g).int().cuda()
    cs = table(400)
    csd, w = cs.cuda(), (1 + 0.1 * torch.randn(512, generator=g)).to(t)
    pos = i32(3, tokens)
    k, kr = torch.zeros(tokens, 1, 512, dtype=t, device="cuda"), torch.zeros(tokens, 1, 64, dtype=t, device="cuda")
    q, qr = torch.zeros(tokens, heads, 512, dtype=t, device="cuda"), torch.zeros(tokens, heads, 64, dtype=t, device="cuda")
    err, wd = i32(1), w.cuda()
    ws = torch.empty(96 << 20, dtype=torch.uint8, device="cuda")
    out = torch.zeros_like(q)
    scale = {} if unit is None else dict(cache_scale=unit)

    def step():
        ql, kvl, left, slots, _ = sfa.page_plan(bt, kv, new, free, count, page_size=page, tokens=tokens, error=err)
        _, turned = sfa.cache_append_slots(cache, slots, pos, k, kr, csd, k_weight=wd, eps=EPS, q_rope=qr, axes=AXES, error=err,
                                           **scale)
        got = sfa.paged_fwd(q, cache, bt, kvl, SCALE, q_rope=turned, layout="TND", act_seq_q=ql, out=out, workspace=ws, **scale)
        kv.copy_(kvl)
        count.copy_(left)
        return turned, got

    graph = None
    if captured:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            res = step()
    history = [torch.zeros(0, 576, dtype=torch.float64) for _ in range(batch)]
    lengths = [0] * batch
    for lens in ([100, 1, 17, 0, 40, 5], [1, 1, 1, 33, 1, 1], [-1, 1, 1, 1, -1, 1], [64, 2, 1, 1, 120, 1], [1, 1, -1, 1, 1, 1]):
        n = sum(max(x, 0) for x in lens)
        rnd = lambda *s: torch.randn(*s, generator=g).to(t)  # noqa: E731
        a, b, c, d = rnd(n, 1, 512), rnd(n, 1, 64), rnd(n, heads, 512), rnd(n, heads, 64)
        at = torch.randint(0, 400, (3, n), generator=g)
        for dst, src in ((k, a), (kr, b), (q, c), (qr, d)):
            dst[:n] = dev(src)
            dst[n:] = float("nan")       # rows of no token
        pos[:, :n] = dev(at.int())
        pos[:, n:] = -5
        new.copy_(torch.tensor(lens, dtype=torch.int32))
        out.fill_(3.0)
        if graph is None:
            res = step()
        else:
            graph.replay()
        torch.cuda.synchronize()
        turned, (got, top, total) = res
        assert err.item() == 0 and sfa.read_device_error(ws) == 0
        assert bool((got[n:] == 3.0).all())
        y = norm(a, w, EPS)[0][:, 0]
        rows = torch.cat((_held(y, unit) if bits == 4 else y, _turn(b, cs, at)[:, 0]), -1)
        first = 0
        for s, m in enumerate(lens):
            if m < 0:
                lengths[s], history[s] = 0, history[s][:0]
                continue
            lengths[s] += m
            history[s] = torch.cat((history[s], rows[first:first + m]))
            keys = history[s]
            if m:
                at_q = slice(first, first + m)
                qq = torch.cat((c[at_q].double(), turned[at_q].cpu().double()), -1)     # as the attention got them
                z = torch.einsum("thd,kd->thk", qq, keys) * SCALE
                j = torch.arange(len(keys))
                z = z.masked_fill((j[None] > len(keys) - m + torch.arange(m)[:, None])[:, None], -math.inf)
                p = z.softmax(-1)
                want = torch.einsum("thk,kd->thd", p, keys[:, :512])
                # a cached row's rotated part (and, of 16 bits, all of it) is one rounding off: a score by u |q| |row|
                # over the roundings' random walk at most, so u times sum |q row|; P as much relatively, twice (sum),
                # and one rounding of its own; values of 16 bits one more
                part = torch.cat((torch.zeros(512) if bits == 4 else torch.ones(512), torch.ones(64))).double()
                dz = (torch.einsum("thd,kd->thk", qq.abs() * part, keys.abs()) * SCALE * (u * 1.01 + 20 * U32)).amax(-1)
                dz = dz + 64 * U32 * SCALE * qq.norm(dim=-1) * keys.norm(dim=-1).max()
                absv = torch.einsum("thk,kd->thd", p, keys[:, :512].abs())
                tol = absv * (u + 2 * dz[..., None].expm1() + 128 * U32 + (0 if bits == 4 else u + 20 * U32)) + \
                    want.abs() * u * 1.01 + floor_of(t) * (1 + len(keys) * keys.abs().max())
                assert bool(((got[at_q].cpu().double() - want).abs() <= tol).all())
                m64 = z.amax(-1)
                assert bool(((top[0, at_q].cpu().double() - m64).abs() <= dz + U32 * (1 + 4 * m64.abs())).all())
            first += m
        assert kv.tolist() == lengths
        assert count.item() == pages - sum(-(-x // page) for x in lengths)
