"""What serving latent attention from a 4-bit cache costs, with what stands
around it: the append that quantises new rows, the attention over them, the
block tables and slot maps of a step, and the position rotation with several
axes (time, height, width) with its gradient.

Every case is what a user's program calls in a step.  With `own` false, `run`
computes the operators in elementary torch operations in 32 bits (64 where a
value is rounded to 4 or 8 bits, so that borders fall alike), rounded once at the
end; with `own` true it calls this repository's package.

A 4-bit row is 416 bytes: 256 of codes (element 2j in the low half of byte j,
2j + 1 in the high one; sign, then 0 .5 1 1.5 2 3 4 6), 32 scales (8 bits, 4 of
exponent and 3 of fraction, one for 16 elements), and 64 rotated elements in 16
bits.  An element is code * scale * 2^scale_exp."""
import math
import random

import torch

own = False

D, DR = 512, 64
ROW, CODES, SCALES = D + DR, D // 2, D // 16
PACKED = CODES + SCALES + 2 * DR
EPS = 1e-6
HEADS = (1, 2, 3, 4, 6, 8, 12, 16, 24, 32, 48, 64, 128)
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}
SOFTMAX_SCALE = 1.0 / math.sqrt(ROW)
VALUES = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
# borders between neighbouring codes; one that lies on a border takes the even code
BORDERS = ((0.25, False), (0.75, True), (1.25, False), (1.75, True), (2.5, False), (3.5, True), (5.0, False))


# ------------------------------------------------------------------ cases
def _attn(name, batch, heads, qmin, qmax, kvmin, kvmax, page, dtype, mode=3, lens=1, scale_exp=0):
    """`batch` sequences with qmin .. qmax new tokens each and kvmin .. kvmax
    tokens in the cache (the new ones among them), drawn with seed `lens`."""
    return dict(name=name, op="attn", batch=batch, heads=heads, qmin=qmin, qmax=qmax, kvmin=kvmin, kvmax=kvmax,
                page=page, dtype=dtype, mode=mode, lens=lens, scale_exp=scale_exp)


def _append(name, batch, heads, qmin, qmax, kvmin, kvmax, page, dtype, by, lens=1, scale_exp=0, interleaved=True):
    """As _attn's; by "table": where the rows go follows from block table and
    lengths; "slots": from a slot map, with positions of three axes."""
    return dict(name=name, op="append", batch=batch, heads=heads, qmin=qmin, qmax=qmax, kvmin=kvmin, kvmax=kvmax,
                page=page, dtype=dtype, by=by, lens=lens, scale_exp=scale_exp, interleaved=interleaved)


def _plan(name, batch, prompts, ended, prompt, kvmax, page, lens=1):
    """A step of `batch` requests: `prompts` of them begin with up to `prompt`
    tokens, `ended` give their pages back, the others have one token more."""
    return dict(name=name, op="plan", batch=batch, prompts=prompts, ended=ended, prompt=prompt, kvmax=kvmax, page=page,
                lens=lens)


def _rope(name, tokens, heads, dtype, grad, sections, mixed, interleaved, table=8192):
    """sections "16,8,8": pairs of each axis; mixed: the axes take turns."""
    return dict(name=name, op="rope", tokens=tokens, heads=heads, dtype=dtype, grad=grad, sections=sections, mixed=mixed,
                interleaved=interleaved, table=table)


def listed():
    return [
        # one short conversation, 16 heads: latency
        _attn("attn4_decode_1x16", 1, 16, 1, 1, 1000, 1000, 64, "bf16"),
        # one token against a long context: the keys are split over the whole GPU
        _attn("attn4_long_1x128", 1, 128, 1, 1, 131071, 131071, 64, "bf16"),
        # a decoding batch with all heads on this GPU
        _attn("attn4_decode_64x128", 64, 128, 1, 1, 1024, 8192, 64, "bf16", lens=2),
        # a decoding batch of a model whose heads are spread over eight GPUs
        _attn("attn4_decode_128x16", 128, 16, 1, 1, 2048, 16384, 128, "fp16", lens=3),
        # a chunk of a prompt behind what is already cached
        _attn("attn4_chunk_512x128", 1, 128, 512, 512, 16384, 16384, 64, "bf16"),
        # one decoding step of 64 short conversations: one row each into the cache, and the cache's values
        _append("append4_decode_64", 64, 128, 1, 1, 60, 300, 64, "bf16", "table"),
        # prompts with images, by a slot map: every row of the cache is new
        _append("append4_prompts_g16", 8, 16, 1025, 2048, 0, 0, 16, "fp16", "slots", scale_exp=-2, interleaved=False),
        # a decoding step of 64 requests: three begin, two end
        _plan("plan_64", 64, 3, 2, 900, 8192, 64),
        # a large step: 1024 requests, 24 long prompts among them
        _plan("plan_1024", 1024, 24, 40, 4096, 16384, 16, lens=4),
        # a short prompt with an image: latency
        _rope("rope_axes_300x16", 300, 16, "bf16", False, "8,12,12", False, False),
        # a training step's 4096 tokens of text and images, 128 heads
        _rope("rope_axes_4096x128", 4096, 128, "bf16", False, "12,10,10", True, True),
        # the gradients of a long step from the attention's dQRope and dKRope; an odd number of tokens
        _rope("rope_axes_grad_16381x64", 16381, 64, "fp16", True, "8,12,12", False, False),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    heads = rng.choice(HEADS)
    dtype = rng.choice(("bf16", "fp16"))
    lens = rng.randrange(1 << 30)
    page = rng.choice((16, 32, 48, 64, 128, 256))
    op = rng.choice(("attn", "attn", "attn", "append", "plan", "rope"))
    if op == "rope":
        a = rng.randint(1, 30)
        b = rng.randint(1, 31 - a)
        return _rope(None, _log(rng, 1, min(16384, (16384 * 64) // heads)), heads, dtype, rng.random() < 0.5,
                     "%d,%d,%d" % (a, b, 32 - a - b), rng.random() < 0.5, rng.random() < 0.5)
    if op == "plan":
        batch = _log(rng, 1, 1024)
        prompts = rng.randint(0, max(1, batch // 4))
        return _plan(None, batch, prompts, rng.randint(0, (batch - prompts) // 2), _log(rng, 1, min(8192, 98304 // max(1, prompts))),
                     _log(rng, 64, min(32768, (1 << 24) // batch)), page, lens)
    scale_exp = rng.randint(-4, 3)
    if op == "append":
        batch = _log(rng, 1, 64)
        qmax = _log(rng, 1, 12288 // batch)
        kvmax = max(qmax, _log(rng, 16, max(17, 16384 // batch)))
        return _append(None, batch, heads, rng.randint(1, qmax), qmax, qmax, kvmax, page, dtype,
                       rng.choice(("table", "slots")), lens, scale_exp, rng.random() < 0.5)
    mode = rng.choice((3, 3, 3, 0))
    if rng.random() < 0.5:                      # single tokens, up to 512k cached ones in all
        batch = _log(rng, 1, 128)
        kvmax = _log(rng, 16, min(131072, (1 << 19) // batch))
        return _attn(None, batch, heads, 1, 1, rng.randint(1, kvmax), kvmax, page, dtype, mode, lens, scale_exp)
    batch = _log(rng, 1, 8)                     # chunks and drafts
    kvmax = _log(rng, 64, 16384)
    qmax = _log(rng, 2, max(2, min(kvmax, (1 << 22) // (heads * batch * max(1, kvmax // 2048)), 512)))
    return _attn(None, batch, heads, rng.randint(1, qmax), qmax, max(qmax, rng.randint(1, kvmax)), max(qmax, kvmax), page,
                 dtype, mode, lens, scale_exp)


def _lengths(case):
    rng = random.Random(case["lens"])
    q = [rng.randint(case["qmin"], case["qmax"]) for _ in range(case["batch"])]
    kv = [max(a, rng.randint(case["kvmin"], case["kvmax"])) for a in q]
    return q, kv


def _requests(case):
    """Tokens in the cache and new tokens (-1: ended) of every request."""
    rng = random.Random(case["lens"])
    kinds = ["prompt"] * case["prompts"] + ["ended"] * case["ended"]
    kinds += ["step"] * (case["batch"] - len(kinds))
    rng.shuffle(kinds)
    kv = [0 if k == "prompt" else rng.randint(1, case["kvmax"]) for k in kinds]
    new = [rng.randint(1, case["prompt"]) if k == "prompt" else -1 if k == "ended" else 1 for k in kinds]
    return kv, new


def _axes(case):
    """The axis of each of the 32 pairs."""
    n = [int(x) for x in case.get("sections", "8,12,12").split(",")]
    if not case.get("mixed"):
        return [a for a, k in enumerate(n) for _ in range(k)]
    left, got, a = list(n), [], 0
    while len(got) < 32:
        if left[a]:
            got.append(a)
            left[a] -= 1
        a = (a + 1) % 3
    return got


# ------------------------------------------------------------------ inputs
def _table(n):
    """(n, 64) fp32: cos of the 32 angles of every position, then sin."""
    freq = 10000.0 ** (-torch.arange(0, DR, 2, dtype=torch.float64, device="cuda") / DR)
    ang = torch.arange(n, dtype=torch.float64, device="cuda")[:, None] * freq
    return torch.cat((ang.cos(), ang.sin()), 1).float()


def _places(n, g, table):
    """(3, n) positions of a prompt: stretches of text, and images of 16 x 20
    patches whose tokens share a time."""
    t = torch.arange(n, device="cuda")
    start = int(torch.randint(0, 1000, (1,), generator=g, device="cuda"))
    image = (t // 320) % 2 == 1
    at, first = t % 320, start + t // 320 * 60
    text = first + at % 60
    pos = torch.stack((torch.where(image, first, text), torch.where(image, first + at // 20, text),
                       torch.where(image, first + at % 20, text)))
    return (pos % table).int().contiguous()


def _quantise(y):
    """Codes and scales of rows (..., 512), in y's precision: the nearest
    8-bit scale to a sixth of 16 elements' largest, the nearest code to element / scale."""
    a = y.abs().unflatten(-1, (SCALES, 16))
    top = a.amax(-1) / 6.0
    exponent = torch.frexp(top)[1] - 1
    step = torch.ldexp(torch.ones_like(top), exponent.clamp(min=-6) - 3)
    scale = ((top / step).round() * step).clamp(max=448.0)
    code = torch.zeros(a.shape, dtype=torch.uint8, device=y.device)
    s = scale[..., None]
    for border, even in BORDERS:
        code += (a >= border * s) if even else (a > border * s)
    code = torch.where(s > 0, code, 0) + 8 * (y.unflatten(-1, (SCALES, 16)) < 0).to(torch.uint8)
    code = code.flatten(-2)
    return code[..., 0::2] + 16 * code[..., 1::2], scale.float().to(torch.float8_e4m3fn).view(torch.uint8)


def _packed(n, t, g, scale_exp):
    """n packed rows as a cache holds them: normed latent rows, rotated keys."""
    pool = min(n, 8192)
    y = torch.randn(pool, D, generator=g, device="cuda") * 2.0 ** -scale_exp
    codes, scales = _quantise(y)
    rope = torch.randn(pool, DR, generator=g, device="cuda").to(t).view(torch.uint8)
    rows = torch.cat((codes, scales, rope), -1)
    return rows[torch.randint(0, pool, (n,), generator=g, device="cuda")]


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    s = dict(case)

    def randn(*shape, scale=1.0):
        return (torch.randn(*shape, generator=g, device="cuda") * scale).to(t)

    def ints(v):
        return torch.tensor(v, dtype=torch.int32, device="cuda")

    if case["op"] == "plan":
        kv, new = _requests(case)
        page = case["page"]
        held = [-(-x // page) for x in kv]
        per = max(-(-(x + max(n, 0)) // page) for x, n in zip(kv, new)) + 2
        grown = sum(-(-(x + max(n, 0)) // page) - h for x, n, h in zip(kv, new, held))
        spare = grown + 8
        order = torch.randperm(sum(held) + spare, generator=g, device="cuda").int()
        before = torch.cumsum(ints([0] + held), 0)
        i = torch.arange(per, device="cuda")[None]
        there = i < ints(held)[:, None]
        bt = torch.where(there, order[torch.where(there, before[:-1, None] + i, 0)], 0)
        free = torch.full_like(order, -1)
        free[:spare] = order[sum(held):]
        s.update(block_table=bt.int().contiguous(), act_kv=ints(kv), new=ints(new), free=free, count=ints([spare]),
                 tokens=sum(max(n, 0) for n in new))
        return s
    t = DTYPES[case["dtype"]]
    heads = case["heads"]
    if case["op"] == "rope":
        n = case["tokens"]
        s["cs"] = _table(case["table"])
        s["pos"] = _places(n, g, case["table"])
        s["k_rope"], s["q_rope"] = randn(n, 1, DR), randn(n, heads, DR)
        s["axes"] = _axes(case)
        s["axis"] = torch.tensor(s["axes"], device="cuda")
        return s
    ql, kl = _lengths(case)
    page = case["page"]
    need = [-(-x // page) for x in kl]
    pages, per = sum(need) + 3, max(need)
    order = torch.randperm(pages, generator=g, device="cuda").int()
    bt = torch.zeros(case["batch"], per, dtype=torch.int32, device="cuda")
    at = 0
    for b, m in enumerate(need):
        bt[b, :m] = order[at:at + m]
        at += m
    tokens = sum(ql)
    s["block_table"], s["act_q"], s["act_kv"] = bt, ints(ql), ints(kl)
    s["cache"] = _packed(pages * page, t, g, case["scale_exp"]).view(pages, page, PACKED)
    s["cache_scale"] = 2.0 ** case["scale_exp"]
    s["q_rope"] = randn(tokens, heads, DR)
    # sequence and position of every new token, as the plain form's indices
    seq = torch.repeat_interleave(torch.arange(len(ql), device="cuda"), s["act_q"].long())
    first = torch.cumsum(s["act_q"].long(), 0) - s["act_q"].long()
    s["seq"], s["within"] = seq, torch.arange(tokens, device="cuda") - first[seq]
    s["at"] = s["act_kv"].long()[seq] - s["act_q"].long()[seq] + s["within"]
    if case["op"] == "append":
        s["cs"] = _table(16384)
        s["k"], s["k_rope"] = randn(tokens, 1, D, scale=1.7), randn(tokens, 1, DR)
        s["k_weight"] = (1 + 0.1 * torch.randn(D, generator=g, device="cuda")).to(t)
        s["q_rope_out"] = torch.empty_like(s["q_rope"])
        s["axes"] = _axes(case)
        s["axis"] = torch.tensor(s["axes"], device="cuda")
        s["slots"] = (bt.long()[seq, s["at"] // page] * page + s["at"] % page).int()
        s["pos"] = _places(tokens, g, 16384) if case["by"] == "slots" else s["at"].int().expand(3, -1).contiguous()
        return s
    s["q"] = randn(tokens, heads, D)
    s["out"] = torch.empty_like(s["q"])
    chunk = case["batch"] * per * page * 2 * ROW if case["qmax"] > 1 else 0
    s["scratch"] = torch.empty((64 << 20) + chunk, dtype=torch.uint8, device="cuda")
    return s


# ------------------------------------------------------------------ plain forms
def _decode(rows, t, scale):
    """Packed rows (..., 416) as fp32 (..., 576)."""
    value = torch.tensor(VALUES + tuple(-v for v in VALUES), device=rows.device)
    codes = rows[..., :CODES]
    x = torch.stack((value[(codes & 15).long()], value[(codes >> 4).long()]), -1).flatten(-2)
    sc = rows[..., CODES:CODES + SCALES].contiguous().view(torch.float8_e4m3fn).float() * scale
    x = (x.unflatten(-1, (SCALES, 16)) * sc[..., None]).flatten(-2)
    return torch.cat((x, rows[..., CODES + SCALES:].contiguous().view(t).float()), -1)


def _rotate(x, cs, pos, axis, interleaved, back=False):
    """(tokens, heads, 64) in fp32, pair i turned by the angle of its axis' position."""
    i = torch.arange(DR // 2, device=x.device)
    row = pos.long()[axis].T                                    # (tokens, 32): the position of each pair
    c = cs[row, i][:, None]
    s = cs[row, DR // 2 + i][:, None] * (-1.0 if back else 1.0)
    x = x.float()
    if interleaved:
        a, b = x[..., 0::2], x[..., 1::2]
        return torch.stack((a * c - b * s, b * c + a * s), -1).flatten(-2)
    a, b = x[..., :DR // 2], x[..., DR // 2:]
    return torch.cat((a * c - b * s, b * c + a * s), -1)


def _run_append(s):
    t, page = s["q_rope"].dtype, s["page"]
    k = s["k"].double()
    y = k * (k.square().mean(-1, keepdim=True) + EPS).rsqrt() * s["k_weight"].double() / s["cache_scale"]
    codes, scales = _quantise(y[:, 0])
    rope = _rotate(s["k_rope"], s["cs"], s["pos"], s["axis"], s["interleaved"])[:, 0].to(t).view(torch.uint8)
    where = s["block_table"].long()[s["seq"], s["at"] // page] * page + s["at"] % page
    if s["by"] == "slots":
        where = s["slots"].long()
    s["cache"].view(-1, PACKED)[where] = torch.cat((codes, scales, rope), -1)
    s["q_rope_out"].copy_(_rotate(s["q_rope"], s["cs"], s["pos"], s["axis"], s["interleaved"]).to(t))
    return {"cache": _decode(s["cache"], t, s["cache_scale"]).to(t), "q_rope": s["q_rope_out"]}


def _run_attn(s):
    """All sequences at once, padded to the longest."""
    t, heads, batch = s["q"].dtype, s["heads"], s["batch"]
    rows = _decode(s["cache"][s["block_table"].long()].flatten(1, 2), t, s["cache_scale"])     # (batch, keys, 576)
    there = torch.arange(rows.shape[1], device="cuda") < s["act_kv"][:, None]
    rows = torch.where(there[..., None], rows, 0.0)
    q = torch.zeros(batch, s["qmax"], heads, ROW, device="cuda")
    q[s["seq"], s["within"]] = torch.cat((s["q"], s["q_rope"]), -1).float()
    x = torch.matmul(q.flatten(1, 2), rows.transpose(1, 2)) * SOFTMAX_SCALE                      # (batch, new * heads, keys)
    x = x.view(batch, s["qmax"], heads, -1)
    last = s["act_kv"][:, None] - 1 + torch.zeros(batch, s["qmax"], dtype=torch.int32, device="cuda")
    if s["mode"] == 3:
        last = s["act_kv"][:, None] - s["act_q"][:, None] + torch.arange(s["qmax"], device="cuda")
        last = torch.minimum(last, s["act_kv"][:, None] - 1)
    see = torch.arange(x.shape[-1], device="cuda") <= last[..., None]
    x.masked_fill_(~see[:, :, None], -math.inf)
    top = x.amax(-1, keepdim=True)
    x.sub_(torch.where(top == -math.inf, 0.0, top)).exp_()
    total = x.sum(-1, keepdim=True)
    o = torch.matmul(x.flatten(1, 2), rows[..., :D]).view(batch, s["qmax"], heads, D)
    o = torch.where(total > 0, o / total, 0.0)
    at = (s["seq"], s["within"])
    return {"out": o[at].to(t), "softmax_max": top[at][None, ..., 0], "softmax_sum": total[at][None, ..., 0]}


def _run_plan(s):
    """Ended requests' pages join the free ones at their end, new pages come
    from there."""
    page, kv, new, bt, free, count = s["page"], s["act_kv"], s["new"], s["block_table"], s["free"], s["count"]
    n, ended = new.clamp(min=0), new < 0
    held = (kv + page - 1) // page
    kv2 = torch.where(ended, 0, kv + n)
    grown = torch.where(ended, 0, (kv2 + page - 1) // page - held)
    back = torch.where(ended, held, 0)
    grown_sum, back_sum = torch.cumsum(grown, 0), torch.cumsum(back, 0)
    i = torch.arange(free.numel(), device="cuda")
    r = i - count
    b = torch.searchsorted(back_sum, r, right=True).clamp(max=kv.numel() - 1)
    r = (r - (back_sum - back)[b]).clamp(0, bt.shape[1] - 1)
    pool = torch.where(i < count, free, bt[b, r])
    total = count + back_sum[-1]
    count2 = total - grown_sum[-1]
    j = torch.arange(bt.shape[1], device="cuda")[None]
    mine = (j >= held[:, None]) & (j < (held + grown)[:, None])
    k = total - 1 - ((grown_sum - grown)[:, None] + j - held[:, None])
    bt.copy_(torch.where(mine, pool[k.clamp(0, pool.numel() - 1)], bt))
    free.copy_(torch.where((i >= count) & (i < count2), pool, free))
    tokens = torch.arange(s["tokens"], device="cuda")
    new_sum = torch.cumsum(n, 0)
    seq = torch.searchsorted(new_sum, tokens, right=True)
    pos = kv[seq] + tokens - (new_sum - n)[seq]
    slots = bt[seq, pos // page] * page + pos % page
    return {"block_table": bt, "free": free, "count": count2.int(), "act_kv": kv2.int(), "act_q": n, "slots": slots.int(),
            "positions": pos.int()}


# ------------------------------------------------------------------ one pass
def run(state):
    s, op = state, state["op"]
    if own:
        import sfa_grad_gb300 as sfa
        if op == "rope" and s["grad"]:
            _, dqr, _, dkr, _, _ = sfa.norm_rope_grad(s["pos"], s["cs"], dk_rope=s["k_rope"], dq_rope=s["q_rope"],
                                                      interleaved=s["interleaved"], axes=s["axes"])
            return {"q_rope": dqr, "k_rope": dkr}
        if op == "rope":
            _, qr, _, kr, _, _ = sfa.norm_rope(s["pos"], s["cs"], k_rope=s["k_rope"], q_rope=s["q_rope"],
                                               interleaved=s["interleaved"], axes=s["axes"])
            return {"q_rope": qr, "k_rope": kr}
        if op == "plan":
            act_q, act_kv, count, slots, pos = sfa.page_plan(s["block_table"], s["act_kv"], s["new"], s["free"],
                                                             s["count"], page_size=s["page"], tokens=s["tokens"])
            return {"block_table": s["block_table"], "free": s["free"], "count": count, "act_kv": act_kv, "act_q": act_q,
                    "slots": slots, "positions": pos}
        if op == "append":
            if s["by"] == "slots":
                sfa.cache_append_slots(s["cache"], s["slots"], s["pos"], s["k"], s["k_rope"], s["cs"],
                                       k_weight=s["k_weight"], eps=EPS, interleaved=s["interleaved"],
                                       q_rope=s["q_rope"], q_rope_out=s["q_rope_out"], axes=s["axes"],
                                       cache_scale=s["cache_scale"])
            else:
                sfa.cache_append(s["cache"], s["block_table"], s["act_kv"], s["k"], s["k_rope"], s["cs"],
                                 k_weight=s["k_weight"], eps=EPS, interleaved=s["interleaved"], q_rope=s["q_rope"],
                                 q_rope_out=s["q_rope_out"], layout="TND", act_seq_q=s["act_q"],
                                 cache_scale=s["cache_scale"])
            return {"cache": sfa.cache_unpack(s["cache"], s["q_rope"].dtype, cache_scale=s["cache_scale"]),
                    "q_rope": s["q_rope_out"]}
        out, top, total = sfa.paged_fwd(s["q"], s["cache"], s["block_table"], s["act_kv"], SOFTMAX_SCALE,
                                        q_rope=s["q_rope"], layout="TND", act_seq_q=s["act_q"], sparse_mode=s["mode"],
                                        out=s["out"], workspace=s["scratch"], cache_scale=s["cache_scale"])
        return {"out": out, "softmax_max": top, "softmax_sum": total}
    if op == "rope":
        return {x: _rotate(s[x], s["cs"], s["pos"], s["axis"], s["interleaved"], s["grad"]).to(s[x].dtype)
                for x in ("q_rope", "k_rope")}
    if op == "plan":
        return _run_plan(s)
    if op == "append":
        return _run_append(s)
    return _run_attn(s)


# ------------------------------------------------------------------ what a pass needs
def work(case):
    if case["op"] == "plan":
        kv, new = _requests(case)
        page = case["page"]
        tokens = sum(max(n, 0) for n in new)
        grown = sum(-(-(x + n) // page) - -(-x // page) for x, n in zip(kv, new) if n > 0)
        back = sum(-(-x // page) for x, n in zip(kv, new) if n < 0)
        # lengths in and out; a page read and written for each that moves; the pages under the new tokens; two maps
        return {"bytes": 4 * (4 * len(kv) + 2 * (grown + back) + len(kv) + 2 * tokens), "flops": 0}
    h = case["heads"]
    if case["op"] == "rope":
        n = case["tokens"]
        # a row of cosines and sines a position, as far as there are that many
        return {"bytes": 2 * 2 * n * DR * (h + 1) + 12 * n + 4 * DR * min(n, case["table"]), "flops": 4 * n * DR * (h + 1)}
    ql, kl = _lengths(case)
    n = sum(ql)
    table = 4 * sum(-(-x // case["page"]) for x in kl) + 8 * len(ql)
    if case["op"] == "append":
        rows = (sum(-(-x // case["page"]) for x in kl) + 3) * case["page"]   # of the cache, unpacked
        return {"bytes": 2 * n * ROW + n * PACKED + 2 * 2 * n * h * DR + 4 * DR * n + 2 * D + table + rows * (PACKED + 2 * ROW),
                "flops": 4 * n * (ROW + h * DR) + rows * D}
    pairs = 0
    for a, b in zip(ql, kl):
        pairs += a * b if case["mode"] == 0 else a * (b - a) + a * (a + 1) // 2
    return {"bytes": PACKED * sum(kl) + 2 * n * h * (ROW + D) + 8 * n * h + table, "flops": 2 * (ROW + D) * h * pairs}


# ------------------------------------------------------------------ the definitions in 64 bits
def _turn64(x, cs, pos, axes, interleaved, sign=1.0):
    """Every pair as a complex number, times exp(+-i angle)."""
    x = x.double()
    half = DR // 2
    pairs = torch.view_as_complex(x.reshape(*x.shape[:-1], half, 2).contiguous()) if interleaved else \
        torch.complex(x[..., :half].contiguous(), x[..., half:].contiguous())
    tab = cs.double()
    turn = torch.stack([torch.complex(tab[pos[a].long(), i], sign * tab[pos[a].long(), half + i])
                        for i, a in enumerate(axes)], -1)
    pairs = pairs * turn[:, None, :]
    if interleaved:
        return torch.view_as_real(pairs).reshape(x.shape)
    return torch.cat((pairs.real, pairs.imag), -1)


def _decode64(rows, t, scale_exp):
    """Packed rows as doubles: both codes of a byte from a table, scales from their bits."""
    one = [v * s for s in (1.0, -1.0) for v in VALUES]
    pair = torch.tensor([[one[b & 15], one[b >> 4]] for b in range(256)], dtype=torch.float64, device=rows.device)
    x = pair[rows[..., :CODES].int()].flatten(-2)
    b = rows[..., CODES:CODES + SCALES].int()
    e, f = (b >> 3) & 15, (b & 7).double()
    sc = torch.where(e == 0, f / 8 * 2.0 ** -6, (1 + f / 8) * torch.exp2(e.double() - 7)) * 2.0 ** scale_exp
    x = x * sc.repeat_interleave(16, -1)
    return torch.cat((x, rows[..., CODES + SCALES:].contiguous().view(t).double()), -1)


def _held64(y, scale_exp):
    """The values a 4-bit row holds for y: each block's scale, then each
    element, to the nearest value of its kind (ties to even)."""
    blocks = (y * 2.0 ** -scale_exp).reshape(*y.shape[:-1], SCALES, 16)
    want = blocks.abs().max(-1, keepdim=True).values / 6
    low = torch.floor(torch.log2(torch.clamp(want, min=2.0 ** -60)))
    low = torch.where(torch.exp2(low) > want, low - 1, low)
    grid = torch.exp2(torch.clamp(low, min=-6) - 3)
    sc = torch.clamp(torch.round(want / grid) * grid, max=448)
    r = torch.where(sc > 0, blocks.abs() / torch.where(sc > 0, sc, 1.0), 0.0)
    g = torch.where(r < 2, 0.5, torch.where(r < 4, 1.0, 2.0))
    r = torch.clamp(torch.round(r / g) * g, max=6)
    return (torch.sign(blocks) * r * sc).reshape(y.shape) * 2.0 ** scale_exp


def exact(case, seed):
    if case["op"] == "plan" or case["op"] == "attn" and work(case)["flops"] > 8e12:
        return None
    s = prepare(case, seed)
    i = case.get("interleaved", True)
    if case["op"] == "rope":
        sign = -1.0 if case["grad"] else 1.0
        return {x: _turn64(s[x], s["cs"], s["pos"], s["axes"], i, sign) for x in ("q_rope", "k_rope")}
    ql, kl = _lengths(case)
    page, t = case["page"], DTYPES[case["dtype"]]
    if case["op"] == "append":
        cache = _decode64(s["cache"], t, case["scale_exp"])
        k = s["k"].double()
        y = torch.einsum("thd,th,d->thd", k, 1.0 / torch.sqrt((k ** 2).sum(-1) / D + EPS), s["k_weight"].double())
        rows = torch.cat((_held64(y, case["scale_exp"]), _turn64(s["k_rope"], s["cs"], s["pos"], s["axes"], i)), -1)
        first = 0
        for b, (a, m) in enumerate(zip(ql, kl)):
            at = torch.arange(m - a, m, device="cuda")
            cache[s["block_table"][b][at // page].long(), at % page] = rows[first:first + a, 0]
            first += a
        return {"cache": cache, "q_rope": _turn64(s["q_rope"], s["cs"], s["pos"], s["axes"], i)}
    outs, tops, sums, first = [], [], [], 0
    for b, (a, m) in enumerate(zip(ql, kl)):
        keys = _decode64(s["cache"][s["block_table"][b].long()].reshape(-1, PACKED)[:m], t, case["scale_exp"])
        step = max(1, (1 << 28) // (case["heads"] * m))
        for lo in range(0, a, step):
            hi = min(a, lo + step)
            q = torch.cat((s["q"][first + lo:first + hi], s["q_rope"][first + lo:first + hi]), -1).double()
            z = torch.einsum("thd,kd->thk", q, keys) * SOFTMAX_SCALE
            if case["mode"] == 3:
                ahead = torch.arange(m, device="cuda")[None] > torch.arange(m - a + lo, m - a + hi, device="cuda")[:, None]
                z = z.masked_fill(ahead[:, None], -math.inf)
            top = z.max(-1).values
            e = torch.exp(z - top[..., None])
            tot = e.sum(-1)
            outs.append(torch.einsum("thk,kd->thd", e, keys[:, :D]) / tot[..., None])
            tops.append(top)
            sums.append(tot)
        first += a
    return {"out": torch.cat(outs), "softmax_max": torch.cat(tops)[None], "softmax_sum": torch.cat(sums)[None]}
