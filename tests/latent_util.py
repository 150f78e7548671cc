"""Plain 64-bit forms of the latent-row operators, and inputs for their tests."""
from __future__ import annotations

import math

import torch

U32 = 2.0 ** -24
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


def half_step(dtype) -> float:
    return torch.finfo(dtype).eps / 2


def floor_of(dtype) -> float:
    """Half the spacing of the type's smallest values."""
    return torch.finfo(dtype).smallest_normal * torch.finfo(dtype).eps / 2


def table(n, device="cpu"):
    freq = 10000.0 ** (-torch.arange(0, 64, 2, dtype=torch.float64) / 64)
    ang = torch.arange(n, dtype=torch.float64)[:, None] * freq
    return torch.cat((ang.cos(), ang.sin()), 1).float().to(device)


def rotate(x, cs, pos, interleaved, back=False):
    """(tokens, heads, 64) turned; padding tokens give zeros."""
    x = x.double()
    ok = (pos >= 0) & (pos < cs.shape[0])
    row = cs.double()[torch.where(ok, pos, 0).long()][:, None]
    c, s = row[..., :32], row[..., 32:] * (-1 if back else 1)
    a, b = (x[..., 0::2], x[..., 1::2]) if interleaved else (x[..., :32], x[..., 32:])
    u, v = a * c - b * s, b * c + a * s
    y = torch.stack((u, v), -1).flatten(-2) if interleaved else torch.cat((u, v), -1)
    return torch.where(ok[:, None, None], y, 0.0)


def norm(x, w, eps):
    x = x.double()
    r = 1 / (x.square().mean(-1) + eps).sqrt()
    return x * r[..., None] * w.double(), r


def paged_inputs(qlens, kvlens, heads, dtype, *, page=64, rope=True, layout="TND", s1=None, extra=0, seed=0,
                 q_scale=1.0, k_scale=1.0, spare=2, device="cuda", poison=True):
    """Random q, a cache with shuffled pages and its block table.  Rows of the
    cache that belong to no token hold NaN, unused table entries are out of
    range.  extra: TND rows behind the last sequence."""
    g = torch.Generator(device="cpu").manual_seed(seed)
    width = 576 if rope else 512
    t = DTYPES[dtype]
    need = [-(-max(k, 0) // page) for k in kvlens]
    pages = sum(need) + spare
    order = torch.randperm(pages, generator=g).int()
    bt = torch.full((len(kvlens), max(need + [1]) + 1), 1 << 30, dtype=torch.int32)
    cache = torch.full((pages * page, width), float("nan") if poison else 0.0, dtype=t)
    at = 0
    for b, n in enumerate(need):
        bt[b, :n] = order[at:at + n]
        at += n
        j = torch.arange(max(kvlens[b], 0))
        rows = bt[b, (j // page)].long() * page + j % page
        cache[rows] = (torch.randn(len(j), width, generator=g) * k_scale).to(t)
    if layout == "BSND":
        lead = (len(qlens), s1)
    else:
        lead = (sum(qlens) + extra,)
    q = (torch.randn(*lead, heads, 512, generator=g) * q_scale).to(t)
    qr = (torch.randn(*lead, heads, 64, generator=g) * q_scale).to(t) if rope else None
    to = lambda x: None if x is None else x.to(device)  # noqa: E731
    return dict(q=to(q), q_rope=to(qr), cache=to(cache.view(pages, page, width)), block_table=to(bt),
                act_seq_kv=to(torch.tensor(kvlens, dtype=torch.int32)),
                act_seq_q=to(torch.tensor(qlens, dtype=torch.int32)))


def paged_ref(x, qlens, kvlens, scale, mode, layout="TND"):
    """64-bit out, max, sum of every row that belongs to a sequence, with the
    bound of the kernel's error (see `paged_bound`).  Yields (index, out, max,
    sum, bound of out, bound of max and relative bound of sum)."""
    page = x["cache"].shape[1]
    dt = x["cache"].dtype
    first = 0
    for b, (a, m) in enumerate(zip(qlens, kvlens)):
        if a == 0:
            continue
        rows = (slice(first, first + a),) if layout == "TND" else (b, slice(0, a))
        first += a
        q = x["q"][rows].double()
        if x["q_rope"] is not None:
            q = torch.cat((q, x["q_rope"][rows].double()), -1)
        j = torch.arange(m, device=q.device)
        keys = x["cache"].flatten(0, 1)[x["block_table"][b][j // page].long() * page + j % page].double()
        s = torch.einsum("thd,kd->thk", q, keys) * scale
        last = m - a + torch.arange(a, device=q.device) if mode == 3 else torch.full((a,), m - 1, device=q.device)
        see = (j[None] <= last[:, None])[:, None].expand_as(s)
        s = torch.where(see, s, -math.inf)
        top = s.amax(-1) if m else torch.full(s.shape[:-1], -math.inf, device=q.device, dtype=torch.float64)
        e = torch.where(see, torch.exp(s - torch.where(top.isinf(), 0, top)[..., None]), 0.0)
        l = e.sum(-1)
        v = keys[:, :512]
        inv = torch.where(l > 0, 1 / l, 0.0)[..., None]
        out = torch.einsum("thk,kd->thd", e, torch.where(v.isfinite(), v, 0.0)) * inv
        absv = torch.einsum("thk,kd->thd", e, torch.where(v.isfinite(), v, 0.0).abs()) * inv
        yield rows, out, top, l, paged_bound(q, keys, out, absv, l, scale, m, dt, top)


def paged_bound(q, keys, out, absv, l, scale, m, dt, top):
    """Errors of the kernel, by its roundings.  d: a score's error, sums of 576
    products in fp32 whose partial sums stay within |q||k|: 64 units of them
    covers any order of accumulation of random terms (sqrt(576) = 24).  P
    carries d and one rounding to dtype (values of fp16 below 2^-14 a fixed
    2^-25), the sum of values 2^-24 for each of its steps, the result one
    rounding to dtype."""
    u = half_step(dt)
    if m == 0:
        z = torch.zeros_like(out)
        return z, torch.zeros_like(l), torch.zeros_like(l)
    knorm = keys.norm(dim=-1)
    big = torch.nan_to_num(knorm, nan=0.0, posinf=0.0).max()
    d = 64 * U32 * abs(scale) * q.norm(dim=-1) * big + 4 * U32 * torch.nan_to_num(top.abs(), posinf=0.0)
    rel = u + 2 * d[..., None] + (64 + m / 16) * U32
    bound = absv * rel + out.abs() * u * 1.01 + floor_of(dt)
    tiny = floor_of(dt) * m * torch.nan_to_num(keys.abs(), nan=0.0, posinf=0.0).max()
    bound = bound + tiny / torch.clamp(l, min=1.0)[..., None]
    return bound, d + U32, 2 * d + (64 + m / 16) * U32
