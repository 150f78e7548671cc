"""Calls over 4-bit rows whose values are unpacked ahead of them: what is unpacked, and how often."""
import pytest
import torch

import sfa_grad_gb300 as sfa
from cache4_util import packed_inputs, packed_rows
from latent_util import DTYPES
from timing_util import in_turns

FILL = 0xA5


def _both(x, dtype, heads, layout="TND", **kw):
    """The call over 4-bit rows and over the values in 16 bits, with a filled workspace; and what lies behind
    the 16-bit call's part of it."""
    t = DTYPES[dtype]
    lead = x["q"].shape[:-2]
    p = sfa.make_paged_params(x["cache"], x["block_table"], x["act_seq_kv"], tokens=lead.numel(), heads=heads,
                              layout=layout, seq=lead[1] if layout == "BSND" else None, act_seq_q=x["act_seq_q"], dtype=t)
    base, whole = sfa.paged_workspace_size(p), sfa.paged4_workspace_size(p)
    assert whole > base     # unpacked ahead
    ws = torch.full((whole,), FILL, dtype=torch.uint8, device="cuda")
    call = lambda cache, **k: sfa.paged_fwd(x["q"], cache, x["block_table"], x["act_seq_kv"], 0.05, q_rope=x["q_rope"],  # noqa: E731
                                            layout=layout, act_seq_q=x["act_seq_q"], workspace=ws, **k, **kw)
    got = call(x["cache"], cache_scale=x["cache_scale"])
    assert sfa.read_device_error(ws) == 0
    left = ws[base:].clone()
    return got, call(sfa.cache_unpack(x["cache"], t, cache_scale=x["cache_scale"])), left


@pytest.mark.gpu
@pytest.mark.parametrize("layout", ["TND", "BSND"])
@pytest.mark.parametrize("spare", [2, 600])
def test_sequences_without_query_rows_stay_packed(spare, layout):
    """One sequence of eight has new tokens: the others' rows are read by nobody, and not unpacked (with 600
    spare pages by table, else by page)."""
    qlens, kvlens, heads = [0] * 8, [3000] * 8, 8
    qlens[5], kvlens[5] = 600, 700
    x = packed_inputs(qlens, kvlens, heads, "bf16", layout=layout, s1=600, spare=spare, seed=4)
    got, want, left = _both(x, "bf16", heads, layout)
    rows = (slice(None),) if layout == "TND" else (5,)
    assert torch.equal(got[0][rows], want[0][rows])
    assert torch.equal(got[1], want[1]) or layout == "BSND"
    # 11 pages of 64 rows of 1152 bytes, and an entry of 4 bytes for each page of tables and cache; a page
    # more for what else may lie there
    entries = x["block_table"].numel() + x["cache"].shape[0]
    assert int((left != FILL).sum()) <= 12 * 64 * 1152 + 4 * entries


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,rope", [("bf16", True), ("fp16", False)])
@pytest.mark.parametrize("page", [16, 48, 256])
def test_shared_pages_of_different_lengths(page, dtype, rope):
    """Forty sequences name the same pages and reach into them by 1 to 700 rows, the longest neither first nor
    last: the values of every row, whoever unpacks it."""
    heads, batch = 4, 40
    kvlens = [1 + (37 * b * b + 11 * b) % 700 for b in range(batch)]
    kvlens[17] = 700
    qlens = [min(k, 1 + 19 * b % 23) for b, k in enumerate(kvlens)]
    qlens[30] = kvlens[30] = 650
    room = 130 * batch - sum(qlens)
    x = packed_inputs(qlens, kvlens, heads, dtype, rope=rope, page=page, extra=room, seed=6)
    own = x["block_table"][17].clone()
    x["block_table"][:] = own
    x["block_table"][3, 0] = x["block_table"][9, -2] = own[0]      # the same page at another place too
    pages = int(-(-700 // page))
    g = torch.Generator().manual_seed(2)
    cache = packed_rows((pages + 1) * page, dtype, g, rope).view(pages + 1, page, -1).cuda()
    x["block_table"][x["block_table"] < x["cache"].shape[0]] %= pages + 1
    x["cache"] = cache
    got, want, _ = _both(x, dtype, heads)
    n = sum(qlens)
    for a, b in zip(got, want):
        a, b = (a[:n], b[:n]) if a.shape[0] > 1 else (a[:, :n], b[:, :n])
        assert torch.equal(a, b)


@pytest.mark.gpu
def test_a_shared_prompt_is_unpacked_once():
    """64 sequences over one history of 16384 rows: little more than the 16-bit call over its values (223 us
    and 192; 337 where each of the 64 unpacked it)."""
    heads, batch, kv = 128, 64, 16384
    g = torch.Generator(device="cuda").manual_seed(8)
    cpu = torch.Generator().manual_seed(8)
    cache = packed_rows(kv, "bf16", cpu, True).view(-1, 64, 416).cuda()
    values = sfa.cache_unpack(cache, torch.bfloat16)
    table = torch.randperm(kv // 64, generator=g, device="cuda").int().expand(batch, -1).contiguous()
    r = lambda *s: torch.randn(*s, generator=g, device="cuda").bfloat16()  # noqa: E731
    q, qr = r(batch, 5, heads, 512), r(batch, 5, heads, 64)
    i32 = lambda v: torch.full((batch,), v, dtype=torch.int32, device="cuda")  # noqa: E731
    p = sfa.make_paged_params(cache, table, i32(kv), tokens=5 * batch, heads=heads, seq=5, act_seq_q=i32(1),
                              dtype=torch.bfloat16)
    kw = dict(q_rope=qr, act_seq_q=i32(1),
              workspace=torch.empty(sfa.paged4_workspace_size(p), dtype=torch.uint8, device="cuda"))
    lens = i32(kv)
    a, b = torch.zeros_like(q), torch.zeros_like(q)
    packed, dense = in_turns(lambda: sfa.paged_fwd(q, cache, table, lens, 0.04, out=a, **kw),
                             lambda: sfa.paged_fwd(q, values, table, lens, 0.04, out=b, **kw), each=5)
    assert torch.equal(a, b)
    assert packed <= 1.4 * dense, (packed, dense)
