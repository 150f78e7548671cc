"""Plain 64-bit forms of the 4-bit rows, and inputs for their tests."""
from __future__ import annotations

import math

import torch

from latent_util import DTYPES, paged_inputs

CODES, SCALES = 256, 32
MAGNITUDES = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def e4m3_values():
    """What each byte stands for as a scale."""
    out = []
    for b in range(256):
        e, f = b >> 3 & 15, b & 7
        v = f / 8 * 2.0 ** -6 if e == 0 else (1 + f / 8) * 2.0 ** (e - 7)
        out.append((math.nan if b & 127 == 127 else v) * (-1 if b & 128 else 1))
    return torch.tensor(out, dtype=torch.float64)


def values(rows, dtype, cache_scale):
    """Rows (..., 288 or 416) as 64-bit values (..., 512 or 576)."""
    rows = rows.cpu()
    table = torch.tensor(MAGNITUDES + tuple(-v for v in MAGNITUDES), dtype=torch.float64)
    codes = rows[..., :CODES].long()
    x = torch.stack((table[codes & 15], table[codes >> 4]), -1).flatten(-2)
    s = e4m3_values()[rows[..., CODES:CODES + SCALES].long()] * cache_scale
    x = (x.unflatten(-1, (SCALES, 16)) * s[..., None]).flatten(-2)
    rope = rows[..., CODES + SCALES:].contiguous().view(dtype).double()
    return torch.cat((x, rope), -1)


def quantise(y):
    """Codes (..., 512) and scale bytes (..., 32) of 64-bit rows, by distance:
    the nearest of all scales to a sixth of the largest, the nearest of all
    codes, ties to the even one."""
    blocks = y.unflatten(-1, (SCALES, 16))
    bad = ~blocks.isfinite().all(-1)
    top = torch.where(bad[..., None], 0.0, blocks.abs()).amax(-1)
    grid = e4m3_values()[:127]
    want = (top / 6).clamp(max=448.0)

    def nearest(v, grid):
        hi = torch.searchsorted(grid, v.contiguous()).clamp(max=len(grid) - 1)
        lo = (hi - 1).clamp(min=0)
        d = (grid[hi] - v) - (v - grid[lo])
        return torch.where((d < 0) | ((d == 0) & (hi % 2 == 0)), hi, lo)

    sc = nearest(want, grid)
    s = grid[sc][..., None]
    r = torch.where(s > 0, blocks.abs() / torch.where(s > 0, s, 1.0), 0.0).clamp(max=6.0)
    r = torch.where(bad[..., None], 0.0, r)
    code = nearest(r, torch.tensor(MAGNITUDES, dtype=torch.float64))
    return code.flatten(-2), torch.where(bad, 127, sc), bad


def split(rows):
    """Codes without signs of zeros told apart (..., 512) as signed halves, and scale bytes."""
    codes = rows.cpu()[..., :CODES].long()
    c = torch.stack((codes & 15, codes >> 4), -1).flatten(-2)
    return c & 7, c >> 3, rows.cpu()[..., CODES:CODES + SCALES].long()


def packed_rows(n, dtype, gen, rope=True, cache_scale=1.0, spread=6.0):
    """Random rows: every code, scales over `spread` octaves."""
    codes = torch.randint(0, 256, (n, CODES), generator=gen, dtype=torch.int32).to(torch.uint8)
    low = 56 - int(4 * spread)
    scales = torch.randint(low, low + int(8 * spread), (n, SCALES), generator=gen, dtype=torch.int32).to(torch.uint8)
    parts = [codes, scales]
    if rope:
        parts.append(torch.randn(n, 64, generator=gen).to(DTYPES[dtype]).view(torch.uint8))
    return torch.cat(parts, -1)


def packed_inputs(qlens, kvlens, heads, dtype, *, rope=True, cache_scale=1.0, seed=0, poison=True, **kw):
    """latent_util.paged_inputs with a cache of 4 bits; rows of no token hold
    scales that are not numbers.  `values`: the same cache's values."""
    x = paged_inputs(qlens, kvlens, heads, dtype, rope=rope, seed=seed, poison=poison, device="cpu", **kw)
    held = ~x["cache"].isnan().any(-1) if poison else torch.ones(x["cache"].shape[:2], dtype=torch.bool)
    g = torch.Generator().manual_seed(seed + 1000)
    n = held.numel()
    rows = packed_rows(n, dtype, g, rope, cache_scale, 3.0).view(*held.shape, -1)
    # sums of 512 products of normal size: most scales near 1/4 of the unit
    bad = torch.full_like(rows, 255)
    cache = torch.where(held[..., None], rows, bad)
    dense = values(cache, DTYPES[dtype], cache_scale).to(DTYPES[dtype])
    x = {k: v if v is None else v.cuda() for k, v in x.items()}
    return dict(x, cache=cache.cuda(), dense=dense.cuda(), cache_scale=cache_scale)
