"""Rows of 4 bits: their values, the append that quantises, and the attention
over them, against forms in 64 bits."""
import ctypes

import pytest
import torch

import sfa_grad_gb300 as sfa
from cache4_util import packed_inputs, packed_rows, quantise, split, values
from latent_util import DTYPES, U32, half_step, norm, paged_ref, rotate, table

SCALE = 576 ** -0.5
EPS = 1e-6


# ------------------------------------------------------------------ refusals
def test_c_entries_refuse():
    from sfa_grad_gb300.latent import CacheParams, PagedParams, RowsParams, _lib
    f, odd, L = ctypes.c_void_p(256), ctypes.c_void_p(258), _lib()
    null, invalid, shape = sfa.SFA_ERR_NULLPTR, sfa.SFA_ERR_PARAM_INVALID, sfa.SFA_ERR_SHAPE
    p = PagedParams(1, 0, 2, 0, 3, 4, 512, 64, 8, 64, 2, SCALE, 3, 1, 0)
    P = ctypes.byref(p)
    fwd = [f] * 10 + [1 << 40, None]
    app = [f, f, f, f, f, f, None, EPS, f, 9, None, None, None, None]
    for scale in (0.0, -1.0, 3.0, 2.0 ** -15, 2.0 ** 5, float("inf"), float("nan")):
        assert L.sfa_paged4_fwd(P, scale, *fwd) == shape
        assert L.sfa_cache4_append(P, scale, *app) == shape
        c = CacheParams(0, 4, 8, 64, 64, scale)
        assert L.sfa_cache4_unpack(ctypes.byref(c), f, f, None) == shape
    for i in (0, 2, 3, 5, 6, 7, 8, 9):
        a = list(fwd)
        a[i] = None
        assert L.sfa_paged4_fwd(P, 1.0, *a) == null, i
    assert L.sfa_paged4_fwd(P, 1.0, *fwd[:10], 1 << 20, None) == invalid      # the workspace is too small
    n = ctypes.c_size_t(0)
    assert L.sfa_paged4_workspace_size(None, ctypes.byref(n)) == null
    assert L.sfa_paged4_workspace_size(P, None) == null
    for i in (0, 1, 2, 3, 4, 5):
        a = list(app)
        a[i] = odd
        assert L.sfa_cache4_append(P, 1.0, *a) == invalid, i
        a[i] = None
        assert L.sfa_cache4_append(P, 1.0, *a) == null, i
    good = dict(dtype=0, bits=4, num_pages=8, page_size=64, Dr=64, scale=1.0)
    for code, over in ((invalid, dict(dtype=2)), (invalid, dict(bits=8)), (invalid, dict(bits=16)), (shape, dict(Dr=32)),
                       (shape, dict(page_size=24)), (shape, dict(page_size=0)), (shape, dict(num_pages=0)),
                       (shape, dict(num_pages=2 ** 30))):
        c = CacheParams(**{**good, **over})
        assert L.sfa_cache4_unpack(ctypes.byref(c), f, f, None) == code, over
    c = ctypes.byref(CacheParams(**good))
    assert L.sfa_cache4_unpack(c, None, f, None) == null and L.sfa_cache4_unpack(c, f, odd, None) == invalid
    r = RowsParams(0, 1, 3, 4, 9, EPS)
    axes = bytes(32)
    # cache, slots, n_axes, axes, positions, k, k_rope, k_weight, cos_sin, q_rope, q_rope_out, error, stream
    slot = [f, f, 1, axes, f, f, f, f, f, f, f, f, None]
    for i, code in ((0, null), (1, null), (4, null), (5, null), (6, null), (8, null), (10, null)):
        a = list(slot)
        a[i] = None
        assert L.sfa_cache_append_slots(c, ctypes.byref(r), *a) == code, i
    for i in (0, 1, 4, 5, 6, 7, 8, 9, 10, 11):
        a = list(slot)
        a[i] = odd
        assert L.sfa_cache_append_slots(c, ctypes.byref(r), *a) == invalid, i
    for n, at in ((0, axes), (5, axes), (1, bytes([1] + [0] * 31)), (3, bytes([0] * 31 + [3]))):
        a = list(slot)
        a[2:4] = n, at
        assert L.sfa_cache_append_slots(c, ctypes.byref(r), *a) == invalid, n
    for code, over in ((invalid, (1, 1, 3, 4, 9, EPS)), (shape, (0, 1, 3, 4, 0, EPS)), (shape, (0, 1, 3, 4, 9, -1.0)),
                       (shape, (0, 1, -1, 4, 9, EPS)), (shape, (0, 1, 3, 129, 9, EPS))):
        q = RowsParams(*over)
        assert L.sfa_cache_append_slots(c, ctypes.byref(q), *slot) == code, over
    assert L.sfa_cache_append_slots(c, None, *slot) == null and L.sfa_cache_append_slots(None, ctypes.byref(r), *slot) == null


def test_binding_refuses():
    cache = torch.zeros(4, 64, 416, dtype=torch.uint8)
    bt, kv = torch.zeros(2, 2, dtype=torch.int32), torch.ones(2, dtype=torch.int32)
    q, qr = torch.zeros(2, 1, 4, 512, dtype=torch.bfloat16), torch.zeros(2, 1, 4, 64, dtype=torch.bfloat16)
    k, kr, cs = q[:, :, :1].contiguous(), qr[:, :, :1].contiguous(), torch.zeros(9, 64)
    with pytest.raises(ValueError, match="416"):
        sfa.paged_fwd(q, cache[..., :400].contiguous(), bt, kv, 1.0, q_rope=qr)
    with pytest.raises(ValueError, match="bfloat16 or float16"):
        sfa.paged_fwd(q.float(), cache, bt, kv, 1.0, q_rope=qr)
    with pytest.raises(ValueError, match="16 bits"):
        sfa.paged_fwd(q, torch.zeros(4, 64, 576, dtype=torch.bfloat16), bt, kv, 1.0, q_rope=qr, cache_scale=1.0)
    with pytest.raises(ValueError, match="q_rope"):
        sfa.paged_fwd(q, cache[..., :288].contiguous(), bt, kv, 1.0, q_rope=qr)
    with pytest.raises(ValueError, match="rope rows"):
        sfa.cache_append(cache[..., :288].contiguous(), bt, kv, k, kr, cs)
    with pytest.raises(ValueError, match="CUDA"):
        sfa.cache_append(cache, bt, kv, k, kr, cs)
    with pytest.raises(ValueError, match="dtype is required"):
        sfa.make_paged_params(cache, bt, kv, tokens=2, heads=4, seq=1)
    assert sfa.make_paged_params(cache, bt, kv, tokens=2, heads=4, seq=1, dtype=torch.float16).Dr == 64
    with pytest.raises(ValueError, match="uint8"):
        sfa.cache_unpack(q[0], torch.bfloat16)
    with pytest.raises(ValueError, match="rows must be"):
        sfa.cache_unpack(cache, torch.float32)
    slots, pos = torch.zeros(2, dtype=torch.int32), torch.zeros(3, 2, dtype=torch.int32)
    k, kr = k[:, 0], kr[:, 0]
    with pytest.raises(ValueError, match="slots"):
        sfa.cache_append_slots(cache, slots[:1], pos[0], k, kr, cs)
    with pytest.raises(ValueError, match="positions"):
        sfa.cache_append_slots(cache, slots, pos, k, kr, cs)
    with pytest.raises(ValueError, match="positions is required"):
        sfa.cache_append_slots(cache, slots, None, k, kr, cs)
    for axes in ([0] * 31, [0] * 31 + [3], [0] * 33):
        with pytest.raises(ValueError, match="axes"):
            sfa.cache_append_slots(cache, slots, pos, k, kr, cs, axes=axes)
    with pytest.raises(ValueError, match="axes given"):
        sfa.cache_append_slots(cache[..., :288].contiguous(), slots, None, k, axes=[0] * 32)


# ------------------------------------------------------------------ values
@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("rope", [True, False])
def test_every_value(dtype, rope):
    """Every code with every scale, in every unit, exactly."""
    t = DTYPES[dtype]
    g = torch.Generator().manual_seed(5)
    rows = packed_rows(256, dtype, g, rope)
    rows[:, :256] = torch.arange(256, dtype=torch.uint8)             # pairs of codes; 8 bytes a block
    first = torch.arange(256)[:, None] + torch.arange(32)[None]      # every scale meets every block
    rows[:, 256:288] = (first % 256).to(torch.uint8)
    cache = rows.view(16, 16, -1)
    for k in range(-14, 5):
        got = sfa.cache_unpack(cache.cuda(), t, cache_scale=2.0 ** k).cpu()
        want = values(cache, t, 2.0 ** k)
        assert got.shape == want.shape
        assert bool((want.isnan() == got.isnan()).all())
        assert torch.equal(got.double().nan_to_num(nan=0.0), want.nan_to_num(nan=0.0)), k


# ------------------------------------------------------------------ append
def _exact_rows(k, w, cache_scale):
    y = k.cpu().double()
    if w is not None:
        y = norm(y, w.cpu(), EPS)[0]
    return y / cache_scale


def _same(rows, y):
    """Packed rows against y's nearest codes and scales."""
    mag, sign, sc = split(rows)
    want, scales, bad = quantise(y)
    assert torch.equal(sc, scales)
    assert torch.equal(mag, want)
    held = (mag > 0)
    assert bool((sign.bool() == (y < 0))[held].all())


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("exponent", [-9, -2, 0, 3])
def test_append_rounds_as_exact_arithmetic(dtype, exponent):
    """60,000 normed rows of any size: some lie so near a border that fp32 takes the wrong side."""
    t, n = DTYPES[dtype], 30000
    g = torch.Generator().manual_seed(11 + exponent)
    k = (torch.randn(n, 1, 512, generator=g) * torch.exp2(torch.randint(-6, 6, (n, 1, 1), generator=g).float())).to(t)
    w = (1 + 0.2 * torch.randn(512, generator=g)).to(t)
    page = 48
    cache = torch.zeros(-(-n // page) + 1, page, 288, dtype=torch.uint8, device="cuda")
    slots = torch.randperm(cache.shape[0] * page, generator=g)[:n].int()
    sfa.cache_append_slots(cache, slots.cuda(), None, k.cuda(), k_weight=w.cuda(), eps=EPS, cache_scale=2.0 ** exponent)
    _same(cache.flatten(0, 1)[slots.long().cuda()], _exact_rows(k[:, 0], w, 2.0 ** exponent))
    left = torch.ones(cache.shape[0] * page, dtype=torch.bool)
    left[slots.long()] = False
    assert not bool(cache.flatten(0, 1)[left.cuda()].any())


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_append_of_ties_and_extremes(dtype):
    """Rows taken as they are: elements halfway between codes and scales, zeros, one element only, the
    type's largest and smallest, infinities and NaN."""
    t = DTYPES[dtype]
    g = torch.Generator().manual_seed(3)
    k = torch.randint(-96, 97, (2000, 512), generator=g).float() / 8     # quarters of codes at scale 2 and less
    k[:, ::16] = (torch.randint(0, 2, (2000, 32), generator=g) * 2 - 1) * torch.tensor([12.0, 12.75, 6.375, 96 / 8])[
        torch.randint(0, 4, (2000, 32), generator=g)]
    k[0] = 0
    k[1] = 0
    k[1, 77] = 1.0
    k[2] = torch.finfo(t).max
    k[3] = -torch.finfo(t).tiny
    k[4] = torch.linspace(-6, 6, 512)
    k[5] *= 2.0 ** -12
    k[6] *= 2.0 ** -14
    k[7] = 2.0 ** -10 * 6
    k[8, 40], k[8, 100], k[8, 511] = float("inf"), -float("inf"), float("nan")
    k = k.to(t)
    n = k.shape[0]
    for exponent in (0, -3):
        cache = torch.full((n // 16, 16, 288), 7, dtype=torch.uint8, device="cuda")
        sfa.cache_append_slots(cache, torch.arange(n, dtype=torch.int32, device="cuda"), None, k[:, None].cuda(),
                               cache_scale=2.0 ** exponent)
        _same(cache.flatten(0, 1), _exact_rows(k, None, 2.0 ** exponent))


@pytest.mark.gpu
@pytest.mark.parametrize("eps", [0.0, 1e-6])
def test_append_norm_at_the_ends_of_the_range(eps):
    """Rows whose squares overflow or vanish in fp32, weights near the type's largest, one that is not finite."""
    t = torch.bfloat16
    g = torch.Generator().manual_seed(4)
    k = torch.randn(8, 512, generator=g) * torch.tensor([1e38, 1e25, 1e-25, 1e-36, 1.0, 1e10, 1e-10, 1.0])[:, None]
    k = k.clamp(-3e38, 3e38).to(t)
    k[7, 9] = float("inf")
    for w in (torch.ones(512), torch.full((512,), 3e38), torch.full((512,), 1e-30),
              torch.cat((torch.ones(500), torch.full((12,), float("nan"))))):
        w = w.to(t)
        cache = torch.zeros(1, 16, 288, dtype=torch.uint8, device="cuda")
        sfa.cache_append_slots(cache, torch.arange(8, dtype=torch.int32, device="cuda"), None, k[:, None].cuda(),
                               k_weight=w.cuda(), eps=eps)
        _same(cache[0, :8], norm(k, w, eps)[0])


@pytest.mark.gpu
def test_append_with_weights_of_any_size():
    """Large weights beside ordinary ones, rows of large values: whichever way a row is rounded, its large
    elements are cut off at the largest value."""
    t, n = torch.bfloat16, 12000
    g = torch.Generator().manual_seed(21)
    k = (torch.randn(n, 1, 512, generator=g) * torch.exp2(torch.randint(-40, 45, (n, 1, 1), generator=g).float())).to(t)
    w = 1 + 0.2 * torch.randn(512, generator=g)
    w[::32] *= torch.exp2(torch.randint(-90, 95, (16,), generator=g).float())
    w[256] = 2.0 ** 58
    w = w.to(t)
    cache = torch.zeros(n // 16, 16, 288, dtype=torch.uint8, device="cuda")
    sfa.cache_append_slots(cache, torch.arange(n, dtype=torch.int32, device="cuda"), None, k.cuda(), k_weight=w.cuda(), eps=EPS)
    _same(cache.flatten(0, 1), _exact_rows(k[:, 0], w, 1.0))
    w = w.clamp(-2.0 ** 59, 2.0 ** 59)
    sfa.cache_append_slots(cache, torch.arange(n, dtype=torch.int32, device="cuda"), None, k.cuda(), k_weight=w.cuda(), eps=EPS)
    _same(cache.flatten(0, 1), _exact_rows(k[:, 0], w, 1.0))


@pytest.mark.gpu
@pytest.mark.parametrize("packed", [True, False])
@pytest.mark.parametrize("interleaved", [True, False])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("axes", [0, 1, 3, 4])
def test_append_by_table_and_by_slots(packed, interleaved, dtype, axes):
    """Both forms write the rows that the formulas give, and nothing else."""
    t, u = DTYPES[dtype], half_step(DTYPES[dtype])
    qlens, kvlens, heads, page = [3, 0, 1, 20, 5], [3, 40, 17, 70, 5], 33, 16
    x = packed_inputs(qlens, kvlens, heads, dtype, page=page, extra=3, seed=axes)
    n = sum(qlens) + 3
    g = torch.Generator().manual_seed(9)
    k, kr = torch.randn(n, 1, 512, generator=g).to(t).cuda(), torch.randn(n, 1, 64, generator=g).to(t).cuda()
    w = (1 + 0.1 * torch.randn(512, generator=g)).to(t).cuda()
    cs, qr = table(100).cuda(), x["q_rope"]
    cache = x["cache"].clone() if packed else x["dense"].nan_to_num(nan=3.0)
    before, unit = cache.clone(), dict(cache_scale=0.25) if packed else {}
    seq = torch.repeat_interleave(torch.arange(5), torch.tensor(qlens))
    at = torch.cat([torch.arange(b - a, b) for a, b in zip(qlens, kvlens)])
    bt = x["block_table"].cpu().long()
    slots = bt[seq, at // page] * page + at % page
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = torch.full_like(qr, 5.0)
    kw = dict(k_weight=w, eps=EPS, interleaved=interleaved, q_rope=qr, q_rope_out=out, error=err, **unit)
    pos = at[None].repeat(max(axes, 1), 1)
    which = torch.zeros(32, dtype=torch.long)
    if axes == 0:
        sfa.cache_append(cache, x["block_table"], x["act_seq_kv"], k, kr, cs, layout="TND", act_seq_q=x["act_seq_q"], **kw)
    else:
        pos = torch.randint(0, 100, (axes, len(at)), generator=g)
        which = torch.randint(0, axes, (32,), generator=g)
        far = torch.cat((slots, torch.full((3,), -1)))
        full = torch.cat((pos, torch.full((axes, 3), 1000)), 1)      # (padding: its positions do not matter)
        p = full if axes > 1 else full[0]
        sfa.cache_append_slots(cache, far.int().cuda(), p.int().cuda().contiguous(), k, kr, cs,
                               axes=which.tolist() if axes > 1 else None, **kw)
    assert err.item() == 0
    rows = cache.flatten(0, 1)[slots.cuda()].cpu()
    m = len(at)
    where = pos[which].T                                               # (tokens, 32): a position a pair
    i = torch.arange(32)
    angle = torch.cat((cs.cpu()[where, i], cs.cpu()[where, 32 + i]), -1)[:, None]

    def turned(x):
        one = rotate(x.cpu(), angle.flatten(0, 1), torch.arange(m), interleaved)
        return one

    want, got = turned(kr[:m])[:, 0], rows[:, -128:].contiguous().view(t).double() if packed else rows[:, 512:].double()
    # two products and a sum in fp32, one rounding
    tol = (kr[:m, 0].cpu().double().abs().amax(-1, keepdim=True)) * 4 * U32 + want.abs() * u * 1.01
    assert bool(((got - want).abs() <= tol).all())
    want, got = turned(qr[:m]), out[:m].cpu().double()
    tol = qr[:m].cpu().double().abs().amax(-1, keepdim=True) * 4 * U32 + want.abs() * u * 1.01
    assert bool(((got - want).abs() <= tol).all())
    assert bool((out[m:] == 5.0).all())
    y = _exact_rows(k[:m, 0], w, 0.25 if packed else 1.0)
    if packed:
        _same(rows, y)
    else:
        assert bool(((rows[:, :512].double() - y).abs() <= y.abs() * (u * 1.01 + 20 * U32)).all())
    left = torch.ones(cache.shape[0] * page, dtype=torch.bool)
    left[slots] = False
    assert torch.equal(cache.flatten(0, 1)[left.cuda()], before.flatten(0, 1)[left.cuda()])


@pytest.mark.gpu
def test_append_errors():
    """A slot behind the cache and a position outside the table are left out and reported."""
    t = torch.bfloat16
    g = torch.Generator().manual_seed(1)
    k, kr = torch.randn(4, 1, 512, generator=g).to(t).cuda(), torch.randn(4, 1, 64, generator=g).to(t).cuda()
    cs = table(50).cuda()
    for slots, pos, code in (([0, 5, 32, 7], [1, 2, 3, 4], 3), ([0, 5, 6, 7], [1, 2, 50, 4], 4), ([0, 5, 6, 7], [1, 2, -1, 4], 4),
                             ([0, 5, 2 ** 31 - 1, 7], [1, 2, 3, 4], 3), ([0, 5, -2 ** 31, 7], [1, 2, 3, 4], 0)):
        cache = torch.zeros(2, 16, 416, dtype=torch.uint8, device="cuda")
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        i = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
        qr = torch.randn(4, 2, 64, generator=g).to(t).cuda()
        _, out = sfa.cache_append_slots(cache, i(slots), i(pos), k, kr, cs, q_rope=qr, q_rope_out=torch.full_like(qr, 9.0),
                                        error=err)
        assert err.item() == code
        written = cache.flatten(0, 1).any(-1).nonzero().flatten().tolist()
        assert written == [0, 5, 7]
        assert bool((out[2] == 9.0).all()) and not bool((out[[0, 1, 3]] == 9.0).all())


# ------------------------------------------------------------------ attention
CASES = {
    # qlens, kvlens, heads, dtype, page, rope, mode, layout, s1, extra
    "one_key": ([1], [1], 1, "bf16", 16, True, 3, "BSND", 1, 0),
    "no_key": ([1, 2, 3], [0, 1, 0], 4, "fp16", 16, True, 3, "TND", None, 0),
    "borders": ([1] * 13, [1, 15, 16, 17, 62, 63, 64, 65, 127, 128, 129, 255, 257], 16, "bf16", 64, True, 3, "TND", None, 3),
    "heads_32": ([1] * 5, [700, 64, 1, 130, 2000], 32, "fp16", 128, True, 3, "BSND", 1, 0),
    "heads_17": ([1, 0, 1, 1], [400, 90, 33, 70], 17, "fp16", 48, True, 3, "TND", None, 2),
    "heads_33": ([1] * 6, [700, 64, 1, 130, 2000, 63], 33, "fp16", 128, True, 3, "BSND", 1, 0),
    "heads_64": ([1] * 5 + [0], [900, 65, 1, 128, 3000, 70], 64, "bf16", 64, True, 3, "TND", None, 1),
    "heads_128": ([1] * 4, [900, 65, 1, 2050], 128, "bf16", 64, True, 3, "BSND", 1, 0),
    "heads_100": ([2, 1, 1], [300, 9, 129], 100, "fp16", 32, True, 3, "BSND", 2, 0),
    "drafts": ([3, 2, 1, 4], [500, 2, 64, 67], 8, "bf16", 32, True, 3, "BSND", 4, 0),
    "more_new_than_cached": ([4, 4], [3, 70], 5, "fp16", 16, True, 3, "BSND", 4, 0),
    "chunk": ([70, 1, 33], [170, 40, 33], 24, "bf16", 64, True, 3, "TND", None, 2),
    "chunk_no_mask": ([20, 9], [30, 300], 64, "fp16", 48, True, 0, "TND", None, 0),
    "uneven": ([60] + [1] * 40, [300] + list(range(1, 41)), 10, "bf16", 64, True, 3, "TND", None, 0),
    "no_mask": ([1, 2], [200, 40], 12, "bf16", 64, True, 0, "TND", None, 0),
    "no_rope": ([1, 2, 1], [500, 129, 3], 16, "bf16", 64, False, 3, "TND", None, 0),
    "no_rope_64": ([1, 1, 1], [500, 129, 3], 50, "fp16", 16, False, 3, "TND", None, 0),
    "large_page": ([1, 1], [1025, 1023], 9, "fp16", 1024, True, 3, "TND", None, 0),
    "long": ([1], [30000], 16, "bf16", 64, True, 3, "BSND", 1, 0),
    "long_128": ([1, 1], [9000, 20], 128, "bf16", 16, True, 3, "TND", None, 0),
    "many": ([1] * 200, [1 + (i * 37) % 300 for i in range(200)], 16, "bf16", 32, True, 3, "BSND", 1, 0),
}


def _inputs(name, **over):
    qlens, kvlens, heads, dtype, page, rope, mode, layout, s1, extra = CASES[name]
    x = packed_inputs(qlens, kvlens, heads, dtype, **{**dict(page=page, rope=rope, layout=layout, s1=s1, extra=extra), **over})
    return x, qlens, kvlens, mode, layout


def _call(x, scale=SCALE, mode=3, layout="TND", **kw):
    return sfa.paged_fwd(x["q"], x["cache"], x["block_table"], x["act_seq_kv"], scale, q_rope=x["q_rope"], layout=layout,
                         act_seq_q=x["act_seq_q"], sparse_mode=mode, cache_scale=x["cache_scale"], **kw)


def _buffers(x, layout):
    q = x["q"]
    st = (q.shape[0], 1, q.shape[1], q.shape[2]) if layout == "BSND" else (1, q.shape[0], q.shape[1])
    f = lambda: torch.full(st, 77.0, device="cuda")  # noqa: E731
    return dict(out=torch.full_like(q, 77.0), softmax_max=f(), softmax_sum=f())


def _check(x, got, qlens, kvlens, scale=SCALE, mode=3, layout="TND"):
    out, top, total = (t.clone() for t in got)
    top, total = (t.squeeze(1 if layout == "BSND" else 0) for t in (top, total))
    ref = dict(x, cache=x["dense"])
    # A weight below 2^-126 is zero (the exponential flushes there), which adds up to 2^-126 x (keys) x (largest value)
    # over the sum.  It shows here only: in 4 bits the values of a row's heavy keys are often exactly zero.
    largest = x["dense"].nan_to_num(nan=0.0).abs().max().double()
    for rows, o, m, l, (bo, bm, bl) in paged_ref(ref, qlens, kvlens, scale, mode, layout):
        bo = bo + 2.0 ** -126 * max(kvlens) * largest / l.clamp(min=1.0)[..., None]
        assert bool(((out[rows].double() - o).abs() <= bo).all())
        seen = l > 0
        assert bool(((top[rows].double() - m).abs() <= bm)[seen].all())
        assert bool(((total[rows].double() - l).abs() <= bl * l)[seen].all())
        assert bool((top[rows][~seen] == -float("inf")).all()) and bool((total[rows][~seen] == 0).all())
        assert bool((out[rows][~seen] == 0).all())
        out[rows], top[rows], total[rows] = 77.0, 77.0, 77.0
    assert bool((out == 77.0).all()) and bool((top == 77.0).all()) and bool((total == 77.0).all())


@pytest.mark.gpu
@pytest.mark.parametrize("name", list(CASES))
def test_attention(name):
    x, qlens, kvlens, mode, layout = _inputs(name)
    _check(x, _call(x, mode=mode, layout=layout, **_buffers(x, layout)), qlens, kvlens, mode=mode, layout=layout)


@pytest.mark.gpu
@pytest.mark.parametrize("name", ["heads_17", "heads_64", "heads_128", "chunk"])
@pytest.mark.parametrize("exponent", [-5, 2])
def test_attention_units(name, exponent):
    x, qlens, kvlens, mode, layout = _inputs(name, cache_scale=2.0 ** exponent)
    scale = SCALE * 2.0 ** -exponent
    _check(x, _call(x, scale, mode, layout, **_buffers(x, layout)), qlens, kvlens, scale, mode, layout)


@pytest.mark.gpu
@pytest.mark.parametrize("name", ["heads_17", "heads_64", "chunk"])
@pytest.mark.parametrize("scale", [0.7, -SCALE, 0.0])
def test_attention_scales(name, scale):
    x, qlens, kvlens, mode, layout = _inputs(name)
    _check(x, _call(x, scale, mode, layout, **_buffers(x, layout)), qlens, kvlens, scale, mode, layout)


@pytest.mark.gpu
@pytest.mark.parametrize("heads", [16, 40, 128])
def test_attention_nan_ahead(heads):
    """Rows of the cache that are not numbers reach only the tokens that see them."""
    qlens, kvlens = [3, 1], [130, 70]
    x = packed_inputs(qlens, kvlens, heads, "bf16")
    clean = _call(x, **_buffers(x, "TND"))[0].clone()
    flat = x["cache"].flatten(0, 1)
    for at, byte in ((128, 256 + 5), (129, 256 + 31)):      # a block's scale: seen by tokens 1 and 2, and by token 2
        flat[x["block_table"][0, at // 64].long() * 64 + at % 64, byte] = 127
    out = _call(x, **_buffers(x, "TND"))[0]
    assert torch.equal(out[0], clean[0]) and torch.equal(out[3], clean[3])
    assert bool(out[1].isnan().any()) and bool(out[2].isnan().any())


@pytest.mark.gpu
@pytest.mark.parametrize("heads", [17, 60, 128])
@pytest.mark.parametrize("page", [-1, -2 ** 31, "num_pages", 2 ** 31 - 1])
def test_bad_page_is_reported_and_reads_as_zeros(heads, page):
    qlens, kvlens = [1, 0, 1, 1], [400, 90, 33, 70]
    x = packed_inputs(qlens, kvlens, heads, "fp16", page=48)
    ws = torch.empty(64 << 20, dtype=torch.uint8, device="cuda")
    want = _call(x, workspace=ws, **_buffers(x, "TND"))[0]
    assert sfa.read_device_error(ws) == 0
    zero = dict(x, cache=torch.cat((x["cache"], torch.zeros_like(x["cache"][:1]))), block_table=x["block_table"].clone())
    zero["block_table"][0, 1] = x["cache"].shape[0]
    zeros = _call(zero, **_buffers(x, "TND"))
    x["block_table"][0, 1] = x["cache"].shape[0] if page == "num_pages" else page
    got = _call(x, workspace=ws, **_buffers(x, "TND"))
    assert sfa.read_device_error(ws) == 3
    assert all(torch.equal(a, b) for a, b in zip(got, zeros))
    assert torch.equal(got[0][1:], want[1:])


@pytest.mark.gpu
@pytest.mark.parametrize("heads", [16, 128])
@pytest.mark.parametrize("which,value", [("act_seq_kv", -1), ("act_seq_kv", 1 << 20), ("act_seq_q", -1), ("act_seq_q", 50)])
def test_bad_lengths_write_nothing(heads, which, value):
    x = packed_inputs([1, 2, 1], [60, 20, 9], heads, "bf16")
    x[which][1] = value
    ws = torch.empty(64 << 20, dtype=torch.uint8, device="cuda")
    got = _call(x, workspace=ws, **_buffers(x, "TND"))
    assert sfa.read_device_error(ws) == 2
    assert all(bool((t == 77.0).all()) for t in got)


@pytest.mark.gpu
@pytest.mark.parametrize("name", ["many", "long_128", "chunk"])
def test_same_bits_and_graph(name):
    """Two calls give the same bits; a graph captured once serves shorter lengths and other pages."""
    x, qlens, kvlens, mode, layout = _inputs(name)
    buf = _buffers(x, layout)
    a = [t.clone() for t in _call(x, mode=mode, layout=layout, **buf)]
    b = _call(x, mode=mode, layout=layout, **_buffers(x, layout))
    assert all(torch.equal(u, v) for u, v in zip(a, b))
    ws = torch.empty(192 << 20, dtype=torch.uint8, device="cuda")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = _call(x, mode=mode, layout=layout, workspace=ws, **buf)
    kvlens = [max(1, q, k // 2) for q, k in zip(qlens, kvlens)]
    x["act_seq_kv"].copy_(torch.tensor(kvlens, dtype=torch.int32))
    for _ in range(2):
        for t in got:
            t.fill_(77.0)
        g.replay()
        torch.cuda.synchronize()
        _check(x, got, qlens, kvlens, mode=mode, layout=layout)
    assert sfa.read_device_error(ws) == 0


@pytest.mark.gpu
@pytest.mark.parametrize("heads", [16, 128])
def test_shared_pages_and_streams(heads):
    """Sequences that share their first pages, on a stream of the caller's, two calls at once."""
    qlens, kvlens, page = [1, 1, 1], [300, 340, 280], 64
    x = packed_inputs(qlens, kvlens, heads, "bf16", page=page, poison=False)
    x["block_table"][1:, :4] = x["block_table"][0, :4]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = [_call(x, stream=s, **_buffers(x, "TND")) for s in streams]
    torch.cuda.synchronize()
    for g in got:
        _check(x, g, qlens, kvlens)


@pytest.mark.gpu
def test_no_token():
    x = packed_inputs([0, 0], [5, 9], 4, "bf16")
    out, top, total = _call(dict(x, q=x["q"][:0], q_rope=x["q_rope"][:0]))
    assert out.numel() == top.numel() == total.numel() == 0
    cache = x["cache"].clone()
    e = torch.empty(0, 1, 512, dtype=torch.bfloat16, device="cuda")
    i = torch.empty(0, dtype=torch.int32, device="cuda")
    sfa.cache_append_slots(cache, i, i, e, e[..., :64].contiguous(), table(9).cuda())
    assert torch.equal(cache, x["cache"])
