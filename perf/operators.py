"""What the latent-attention operators around the sparse attention cost: the
position rotation and norms of queries and keys with their gradients, the
append to a paged cache of latent rows, and the attention of new tokens over
that cache.

Every case is one call a user's program makes.  With `own` false, `run`
computes the operator in elementary torch operations in 32 bits, rounded once
at the end; with `own` true it calls this repository's package."""
import math
import random

import torch

own = False

D, DR = 512, 64
ROW = D + DR
EPS = 1e-6
HEADS = (1, 2, 3, 4, 6, 8, 12, 16, 24, 32, 48, 64, 128)
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}
SCALE = 1.0 / math.sqrt(ROW)


# ------------------------------------------------------------------ cases
def _norm(name, op, tokens, heads, qnorm, dtype, interleaved, table):
    return dict(name=name, op=op, tokens=tokens, heads=heads, qnorm=qnorm, dtype=dtype, interleaved=interleaved,
                table=table)


def _paged(name, op, batch, heads, qmin, qmax, kvmin, kvmax, page, dtype, mode=3, lens=1, interleaved=True):
    """`batch` sequences with qmin .. qmax new tokens each and kvmin .. kvmax
    tokens in the cache (the new ones among them), drawn with seed `lens`."""
    return dict(name=name, op=op, batch=batch, heads=heads, qmin=qmin, qmax=qmax, kvmin=kvmin, kvmax=kvmax, page=page,
                dtype=dtype, mode=mode, lens=lens, interleaved=interleaved)


def listed():
    return [
        # a short prompt's rows: latency
        _norm("rope_norm_16", "norm_rope", 16, 4, False, "bf16", True, 4096),
        # a training step's 4096 tokens with 128 heads: latent keys normalised, queries and keys rotated
        _norm("rope_norm_4096x128", "norm_rope", 4096, 128, False, "bf16", True, 4096),
        # the gradients of the same step, from the attention's dQRope, dK and dKRope
        _norm("rope_norm_grad_4096x128", "norm_rope_grad", 4096, 128, False, "bf16", True, 4096),
        # few heads, each query head normalised too; long sequences; an odd number of tokens
        _norm("rope_norm_grad_q16", "norm_rope_grad", 16381, 16, True, "fp16", False, 32768),
        # one decoding step of 64 sequences: one row each into the cache
        _paged("append_decode_64", "append", 64, 128, 1, 1, 1000, 8192, 64, "bf16"),
        # prompts cut into chunks of up to 2048 tokens
        _paged("append_chunk_g64", "append", 8, 64, 1025, 2048, 2048, 16384, 16, "bf16", interleaved=False),
        # one short conversation, 16 heads: latency
        _paged("decode_1x16", "paged", 1, 16, 1, 1, 1000, 1000, 64, "bf16"),
        # one token against a long context: the keys are split over the whole GPU
        _paged("decode_long_1x128", "paged", 1, 128, 1, 1, 131071, 131071, 64, "bf16"),
        # a decoding batch with all heads on this GPU
        _paged("decode_64x128", "paged", 64, 128, 1, 1, 1024, 8192, 64, "bf16", lens=2),
        # a decoding batch of a model whose heads are spread over eight GPUs
        _paged("decode_128x16", "paged", 128, 16, 1, 1, 2048, 16384, 128, "fp16", lens=3),
        # a chunk of a prompt behind what is already cached
        _paged("chunk_512x128", "paged", 1, 128, 512, 512, 16384, 16384, 64, "bf16"),
        # chunks and drafted tokens of several sequences in one batch
        _paged("mixed_g64", "paged", 6, 64, 1, 300, 700, 9000, 32, "fp16", lens=5),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    heads = rng.choice(HEADS)
    dtype = rng.choice(("bf16", "fp16"))
    inter = rng.random() < 0.5
    op = rng.choice(("norm_rope", "norm_rope_grad", "append", "paged", "paged", "paged"))
    if op.startswith("norm"):
        qnorm = rng.random() < 0.4
        most = (4096 * 128) // (heads * (8 if qnorm else 1))
        return _norm(None, op, _log(rng, 1, max(1, min(16384, most))), heads, qnorm, dtype, inter, 32768)
    page = rng.choice((16, 32, 48, 64, 128, 256))
    lens = rng.randrange(1 << 30)
    if op == "append":
        batch = _log(rng, 1, 128)
        qmax = _log(rng, 1, max(1, 16384 // batch))
        kvmax = max(qmax, _log(rng, 64, 16384))
        return _paged(None, op, batch, heads, rng.randint(1, qmax), qmax, qmax, kvmax, page, dtype, 3, lens, inter)
    mode = rng.choice((3, 3, 3, 0))
    if rng.random() < 0.5:                      # single tokens, up to 512k cached ones in all
        batch = _log(rng, 1, 128)
        kvmax = _log(rng, 16, min(131072, (1 << 19) // batch))
        return _paged(None, op, batch, heads, 1, 1, rng.randint(1, kvmax), kvmax, page, dtype, mode, lens)
    batch = _log(rng, 1, 8)                     # chunks and drafts
    kvmax = _log(rng, 64, 16384)
    qmax = _log(rng, 2, max(2, min(kvmax, (1 << 22) // (heads * batch * max(1, kvmax // 2048)), 512)))
    return _paged(None, op, batch, heads, rng.randint(1, qmax), qmax, max(qmax, rng.randint(1, kvmax)),
                  max(qmax, kvmax), page, dtype, mode, lens)


def _lengths(case):
    rng = random.Random(case["lens"])
    q = [rng.randint(case["qmin"], case["qmax"]) for _ in range(case["batch"])]
    kv = [max(a, rng.randint(case["kvmin"], case["kvmax"])) for a in q]
    return q, kv


# ------------------------------------------------------------------ inputs
def _table(n):
    """(n, 64) fp32: cos of the 32 angles of every position, then sin."""
    freq = 10000.0 ** (-torch.arange(0, DR, 2, dtype=torch.float64, device="cuda") / DR)
    ang = torch.arange(n, dtype=torch.float64, device="cuda")[:, None] * freq
    return torch.cat((ang.cos(), ang.sin()), 1).float()


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    t = DTYPES[case["dtype"]]
    heads = case["heads"]

    def randn(*shape, scale=1.0):
        return (torch.randn(*shape, generator=g, device="cuda") * scale).to(t)

    s = dict(case)
    if case["op"].startswith("norm"):
        n = case["tokens"]
        s["cs"] = _table(case["table"])
        # packed sequences: positions restart at the sequences' beginnings
        start = int(torch.randint(0, max(1, case["table"] - n), (1,), generator=g, device="cuda"))
        s["pos"] = ((start + torch.arange(n, device="cuda")) % case["table"]).int()
        s["k"], s["k_rope"], s["q_rope"] = randn(n, 1, D, scale=1.7), randn(n, 1, DR), randn(n, heads, DR)
        s["k_weight"] = (1 + 0.1 * torch.randn(D, generator=g, device="cuda")).to(t)
        s["q"] = s["q_weight"] = None
        if case["qnorm"]:
            s["q"] = randn(n, heads, D, scale=0.8)
            s["q_weight"] = (1 + 0.1 * torch.randn(D, generator=g, device="cuda")).to(t)
        if case["op"] == "norm_rope_grad":
            # what the forward saved, and the attention's gradients
            s["k_rstd"] = (s["k"].float().square().mean(-1) + EPS).rsqrt()
            s["q_rstd"] = (s["q"].float().square().mean(-1) + EPS).rsqrt() if case["qnorm"] else None
            s["dk"], s["dk_rope"], s["dq_rope"] = randn(n, 1, D), randn(n, 1, DR), randn(n, heads, DR)
            s["dq"] = randn(n, heads, D) if case["qnorm"] else None
        return s
    ql, kl = _lengths(case)
    page = case["page"]
    per = max(-(-x // page) for x in kl)
    need = [-(-x // page) for x in kl]
    pages = sum(need) + 3
    order = torch.randperm(pages, generator=g, device="cuda").int()
    bt = torch.zeros(case["batch"], per, dtype=torch.int32, device="cuda")
    at = 0
    for b, m in enumerate(need):
        bt[b, :m] = order[at:at + m]
        at += m
    tokens = sum(ql)
    s["block_table"] = bt
    s["act_q"] = torch.tensor(ql, dtype=torch.int32, device="cuda")
    s["act_kv"] = torch.tensor(kl, dtype=torch.int32, device="cuda")
    s["cache"] = randn(pages, page, ROW)
    s["q_rope"] = randn(tokens, heads, DR)
    # sequence and position of every new token, as the plain form's indices
    seq = torch.repeat_interleave(torch.arange(len(ql), device="cuda"), s["act_q"].long())
    first = torch.cumsum(s["act_q"].long(), 0) - s["act_q"].long()
    s["seq"], s["within"] = seq, torch.arange(tokens, device="cuda") - first[seq]
    s["pos"] = s["act_kv"].long()[seq] - s["act_q"].long()[seq] + s["within"]
    if case["op"] == "append":
        s["cs"] = _table(16384)
        s["k"], s["k_rope"] = randn(tokens, 1, D, scale=1.7), randn(tokens, 1, DR)
        s["k_weight"] = (1 + 0.1 * torch.randn(D, generator=g, device="cuda")).to(t)
        s["q_rope_out"] = torch.empty_like(s["q_rope"])
    else:
        s["q"] = randn(tokens, heads, D)
        s["out"] = torch.empty_like(s["q"])
        s["scratch"] = torch.empty(64 << 20, dtype=torch.uint8, device="cuda")
    return s


# ------------------------------------------------------------------ plain forms
def _rotate(x, cs, pos, interleaved, back=False):
    """(tokens, heads, 64) in fp32, turned by every token's angles."""
    c = cs[pos.long(), :DR // 2][:, None]
    s = cs[pos.long(), DR // 2:][:, None] * (-1.0 if back else 1.0)
    x = x.float()
    if interleaved:
        a, b = x[..., 0::2], x[..., 1::2]
        return torch.stack((a * c - b * s, b * c + a * s), -1).flatten(-2)
    a, b = x[..., :DR // 2], x[..., DR // 2:]
    return torch.cat((a * c - b * s, b * c + a * s), -1)


def _norm_plain(x, w):
    x = x.float()
    r = (x.square().mean(-1, keepdim=True) + EPS).rsqrt()
    return x * r * w.float(), r[..., 0]


def _norm_grad_plain(x, w, r, dy):
    x, dy, r = x.float(), dy.float(), r[..., None]
    g = dy * w.float()
    dx = r * (g - x * (r * r) * (g * x).mean(-1, keepdim=True))
    return dx, (dy * (x * r)).flatten(0, 1).sum(0)


def _run_norm_rope(s):
    t, q, rq = s["k"].dtype, None, None
    if s["q"] is not None:
        q, rq = _norm_plain(s["q"], s["q_weight"])
        q = q.to(t)
    k, rk = _norm_plain(s["k"], s["k_weight"])
    return {"q": q, "q_rope": _rotate(s["q_rope"], s["cs"], s["pos"], s["interleaved"]).to(t), "k": k.to(t),
            "k_rope": _rotate(s["k_rope"], s["cs"], s["pos"], s["interleaved"]).to(t), "q_rstd": rq, "k_rstd": rk}


def _run_norm_rope_grad(s):
    t, dq, dwq = s["k"].dtype, None, None
    if s["q"] is not None:
        dq, dwq = _norm_grad_plain(s["q"], s["q_weight"], s["q_rstd"], s["dq"])
        dq = dq.to(t)
    dk, dwk = _norm_grad_plain(s["k"], s["k_weight"], s["k_rstd"], s["dk"])
    return {"dq": dq, "dq_rope": _rotate(s["dq_rope"], s["cs"], s["pos"], s["interleaved"], True).to(t),
            "dk": dk.to(t), "dk_rope": _rotate(s["dk_rope"], s["cs"], s["pos"], s["interleaved"], True).to(t),
            "dq_weight": dwq, "dk_weight": dwk}


def _run_append(s):
    t, page = s["cache"].dtype, s["page"]
    k, _ = _norm_plain(s["k"], s["k_weight"])
    row = torch.cat((k, _rotate(s["k_rope"], s["cs"], s["pos"], s["interleaved"])), -1)[:, 0].to(t)
    where = s["block_table"].long()[s["seq"], s["pos"] // page] * page + s["pos"] % page
    s["cache"].view(-1, ROW)[where] = row
    s["q_rope_out"].copy_(_rotate(s["q_rope"], s["cs"], s["pos"], s["interleaved"]).to(t))
    return {"cache": s["cache"], "q_rope": s["q_rope_out"]}


def _run_paged(s):
    """All sequences at once, padded to the longest."""
    t, heads, batch = s["q"].dtype, s["heads"], s["batch"]
    rows = s["cache"][s["block_table"].long()].flatten(1, 2).float()            # (batch, keys, 576)
    there = torch.arange(rows.shape[1], device="cuda") < s["act_kv"][:, None]
    rows = torch.where(there[..., None], rows, 0.0)
    q = torch.zeros(batch, s["qmax"], heads, ROW, device="cuda")
    q[s["seq"], s["within"]] = torch.cat((s["q"], s["q_rope"]), -1).float()
    x = torch.matmul(q.flatten(1, 2), rows.transpose(1, 2)) * SCALE               # (batch, new * heads, keys)
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


# ------------------------------------------------------------------ one pass
def run(state):
    s, op = state, state["op"]
    if own:
        import sfa_grad_gb300 as sfa
        if op == "norm_rope":
            q, qr, k, kr, rq, rk = sfa.norm_rope(s["pos"], s["cs"], k=s["k"], k_weight=s["k_weight"],
                                                 k_rope=s["k_rope"], q=s["q"], q_weight=s["q_weight"],
                                                 q_rope=s["q_rope"], eps=EPS, interleaved=s["interleaved"])
            return {"q": q, "q_rope": qr, "k": k, "k_rope": kr, "q_rstd": rq, "k_rstd": rk}
        if op == "norm_rope_grad":
            dq, dqr, dk, dkr, dwq, dwk = sfa.norm_rope_grad(
                s["pos"], s["cs"], k=s["k"], k_weight=s["k_weight"], k_rstd=s["k_rstd"], dk=s["dk"],
                dk_rope=s["dk_rope"], q=s["q"], q_weight=s["q_weight"], q_rstd=s["q_rstd"], dq=s["dq"],
                dq_rope=s["dq_rope"], interleaved=s["interleaved"])
            return {"dq": dq, "dq_rope": dqr, "dk": dk, "dk_rope": dkr, "dq_weight": dwq, "dk_weight": dwk}
        if op == "append":
            sfa.cache_append(s["cache"], s["block_table"], s["act_kv"], s["k"], s["k_rope"], s["cs"],
                             k_weight=s["k_weight"], eps=EPS, interleaved=s["interleaved"], q_rope=s["q_rope"],
                             q_rope_out=s["q_rope_out"], layout="TND", act_seq_q=s["act_q"])
            return {"cache": s["cache"], "q_rope": s["q_rope_out"]}
        out, top, total = sfa.paged_fwd(s["q"], s["cache"], s["block_table"], s["act_kv"], SCALE, q_rope=s["q_rope"],
                                        layout="TND", act_seq_q=s["act_q"], sparse_mode=s["mode"], out=s["out"],
                                        workspace=s["scratch"])
        return {"out": out, "softmax_max": top, "softmax_sum": total}
    if op == "norm_rope":
        return _run_norm_rope(s)
    if op == "norm_rope_grad":
        return _run_norm_rope_grad(s)
    if op == "append":
        return _run_append(s)
    return _run_paged(s)


# ------------------------------------------------------------------ what a pass needs
def work(case):
    h = case["heads"]
    if case["op"].startswith("norm"):
        n = case["tokens"]
        rows = D + DR + h * DR + (h * D if case["qnorm"] else 0)
        rstd = 4 * n * (1 + (h if case["qnorm"] else 0))
        fixed = n * (4 + 4 * DR) + 2 * D
        if case["op"] == "norm_rope":
            return {"bytes": 2 * 2 * n * rows + rstd + fixed, "flops": 4 * n * rows}
        normed = D * (1 + (h if case["qnorm"] else 0))
        return {"bytes": 2 * n * (2 * rows + normed) + rstd + fixed + 4 * D, "flops": 8 * n * rows}
    ql, kl = _lengths(case)
    n = sum(ql)
    table = 4 * sum(-(-x // case["page"]) for x in kl) + 8 * len(ql)
    if case["op"] == "append":
        return {"bytes": 2 * 2 * n * (ROW + h * DR) + 4 * DR * n + table + 2 * D, "flops": 4 * n * (ROW + h * DR)}
    pairs = 0
    for a, b in zip(ql, kl):
        pairs += a * b if case["mode"] == 0 else a * (b - a) + a * (a + 1) // 2
    return {"bytes": 2 * ROW * sum(kl) + 2 * n * h * (ROW + D) + 8 * n * h + table,
            "flops": 2 * (ROW + D) * h * pairs}


# ------------------------------------------------------------------ the definitions in 64 bits
def _turn64(x, cs, pos, interleaved, sign=1.0):
    """Every pair as a complex number, times exp(+-i angle)."""
    x = x.double()
    half = DR // 2
    pairs = torch.view_as_complex(x.reshape(*x.shape[:-1], half, 2).contiguous()) if interleaved else \
        torch.complex(x[..., :half].contiguous(), x[..., half:].contiguous())
    tab = cs.double()[pos.long()]
    pairs = pairs * torch.complex(tab[:, :half].contiguous(), sign * tab[:, half:].contiguous())[:, None, :]
    if interleaved:
        return torch.view_as_real(pairs).reshape(x.shape)
    return torch.cat((pairs.real, pairs.imag), -1)


def _rms64(x, w):
    x = x.double()
    r = 1.0 / torch.sqrt((x ** 2).sum(-1) / D + EPS)
    return torch.einsum("thd,th,d->thd", x, r, w.double()), r


def _rms64_grad(x, w, r, dy):
    x, w, r, dy = x.double(), w.double(), r.double(), dy.double()
    inner = torch.einsum("thd,thd,d->th", dy, x, w) / D
    dx = torch.einsum("thd,d,th->thd", dy, w, r) - torch.einsum("thd,th->thd", x, inner * r ** 3)
    return dx, torch.einsum("thd,thd,th->d", dy, x, r)


def exact(case, seed):
    if case["op"] == "paged" and work(case)["flops"] > 8e12:
        return None
    s = prepare(case, seed)
    op, i = case["op"], case["interleaved"]
    if op == "norm_rope":
        q, rq = _rms64(s["q"], s["q_weight"]) if case["qnorm"] else (None, None)
        k, rk = _rms64(s["k"], s["k_weight"])
        return {"q": q, "q_rope": _turn64(s["q_rope"], s["cs"], s["pos"], i), "k": k,
                "k_rope": _turn64(s["k_rope"], s["cs"], s["pos"], i), "q_rstd": rq, "k_rstd": rk}
    if op == "norm_rope_grad":
        dq, dwq = _rms64_grad(s["q"], s["q_weight"], s["q_rstd"], s["dq"]) if case["qnorm"] else (None, None)
        dk, dwk = _rms64_grad(s["k"], s["k_weight"], s["k_rstd"], s["dk"])
        return {"dq": dq, "dq_rope": _turn64(s["dq_rope"], s["cs"], s["pos"], i, -1.0), "dk": dk,
                "dk_rope": _turn64(s["dk_rope"], s["cs"], s["pos"], i, -1.0), "dq_weight": dwq, "dk_weight": dwk}
    ql, kl = _lengths(case)
    page = case["page"]
    if op == "append":
        cache = s["cache"].double()
        k, _ = _rms64(s["k"], s["k_weight"])
        kr = _turn64(s["k_rope"], s["cs"], s["pos"], i)
        t = 0
        for b, (a, m) in enumerate(zip(ql, kl)):
            at = torch.arange(m - a, m, device="cuda")
            pg = s["block_table"][b][at // page].long()
            cache[pg, at % page, :D] = k[t:t + a, 0]
            cache[pg, at % page, D:] = kr[t:t + a, 0]
            t += a
        return {"cache": cache, "q_rope": _turn64(s["q_rope"], s["cs"], s["pos"], i)}
    outs, tops, sums, t = [], [], [], 0
    for b, (a, m) in enumerate(zip(ql, kl)):
        keys = s["cache"][s["block_table"][b].long()].reshape(-1, ROW)[:m].double()
        step = max(1, (1 << 28) // (case["heads"] * m))
        for lo in range(0, a, step):
            hi = min(a, lo + step)
            q = torch.cat((s["q"][t + lo:t + hi], s["q_rope"][t + lo:t + hi]), -1).double()
            z = torch.einsum("thd,kd->thk", q, keys) * SCALE
            if case["mode"] == 3:
                ahead = torch.arange(m, device="cuda")[None] > torch.arange(m - a + lo, m - a + hi, device="cuda")[:, None]
                z = z.masked_fill(ahead[:, None], -math.inf)
            top = z.max(-1).values
            e = torch.exp(z - top[..., None])
            tot = e.sum(-1)
            outs.append(torch.einsum("thk,kd->thd", e, keys[:, :D]) / tot[..., None])
            tops.append(top)
            sums.append(tot)
        t += a
    return {"out": torch.cat(outs), "softmax_max": torch.cat(tops)[None], "softmax_sum": torch.cat(sums)[None]}
