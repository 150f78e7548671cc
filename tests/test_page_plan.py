"""Block tables and slot maps of a step against a simulation of the requests."""
import ctypes
import random

import pytest
import torch

import sfa_grad_gb300 as sfa


class Pool:
    """Requests and pages as a program on the host would keep them."""

    def __init__(self, batch, max_pages, num_pages, page, seed=0):
        self.rng = random.Random(seed)
        self.page, self.max_pages, self.num_pages = page, max_pages, num_pages
        self.table = [[-7] * max_pages for _ in range(batch)]
        self.kv = [0] * batch
        self.free = list(range(num_pages))
        self.rng.shuffle(self.free)

    def held(self, n):
        return -(-n // self.page)

    def tensors(self):
        i = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
        return dict(block_table=i(self.table), act_seq_kv=i(self.kv),
                    free_pages=i(self.free + [-3] * (self.num_pages - len(self.free))), free_count=i([len(self.free)]))

    def step(self, new):
        """The outputs of a step, by the rules of sfa_page_plan."""
        for b, n in enumerate(new):
            if n < 0:
                self.free += self.table[b][:self.held(self.kv[b])]
        slots, pos = [], []
        for b, n in enumerate(new):
            if n < 0:
                self.kv[b] = 0
                continue
            for j in range(self.held(self.kv[b]), self.held(self.kv[b] + n)):
                self.table[b][j] = self.free.pop()
            for p in range(self.kv[b], self.kv[b] + n):
                slots.append(self.table[b][p // self.page] * self.page + p % self.page)
                pos.append(p)
            self.kv[b] += n
        return [max(n, 0) for n in new], list(self.kv), len(self.free), slots, pos


def _plan(t, new, page, tokens, **kw):
    return sfa.page_plan(t["block_table"], t["act_seq_kv"], torch.tensor(new, dtype=torch.int32, device="cuda"),
                         t["free_pages"], t["free_count"], page_size=page, tokens=tokens, **kw)


def _same(t, got, want, pool, tokens):
    q, kv, count, slots, pos = want
    pad = [-1] * (tokens - len(slots))
    assert got[0].tolist() == q and got[1].tolist() == kv and got[2].tolist() == [count]
    assert got[3].tolist() == slots + pad and got[4].tolist() == pos + pad
    assert t["block_table"].tolist() == pool.table
    assert t["free_pages"].tolist()[:count] == pool.free


@pytest.mark.gpu
@pytest.mark.parametrize("batch,max_pages,page,longest", [(1, 40, 16, 200), (3, 9, 64, 90), (64, 30, 32, 400), (511, 5, 16, 40),
                                                          (1025, 12, 48, 300), (8192, 2, 16, 9)])
def test_steps(batch, max_pages, page, longest):
    """Requests that begin, wait, go on and end, step after step."""
    pool = Pool(batch, max_pages, batch * max_pages, page, seed=batch)
    rng = random.Random(batch)
    t = pool.tensors()
    for step in range(6):
        new = []
        for b in range(batch):
            if pool.kv[b] == 0:
                new.append(rng.choice((0, 1, rng.randint(1, longest))))
            else:
                new.append(rng.choice((-1, 0, 1, 1, 1, rng.randint(2, longest // 2), -5)))
            new[-1] = min(new[-1], max_pages * page - pool.kv[b])
        tokens = sum(max(n, 0) for n in new) + rng.choice((0, 0, 13))
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        got = _plan(t, new, page, tokens, error=err)
        want = pool.step(new)
        _same(t, got, want, pool, tokens)
        assert err.item() == 0
        t.update(act_seq_kv=got[1], free_count=got[2])


@pytest.mark.gpu
def test_all_end_and_the_last_page():
    pool = Pool(5, 4, 20, 16)
    t = pool.tensors()
    for new in ([64] * 5, [-1] * 5, [64, 64, 64, 64, 63], [0, -1, 0, 0, 1], [0] * 5):
        tokens = sum(max(n, 0) for n in new)
        got = _plan(t, new, 16, tokens)
        _same(t, got, pool.step(new), pool, tokens)
        t.update(act_seq_kv=got[1], free_count=got[2])


@pytest.mark.gpu
@pytest.mark.parametrize("what", ["negative", "table", "ended_table", "tokens", "pool", "count", "count_low", "returned"])
def test_a_step_that_does_not_fit_changes_nothing(what):
    pool = Pool(300, 4, 1210, 16, seed=2)
    t = pool.tensors()
    first = [1 + b % 60 for b in range(300)]
    got = _plan(t, first, 16, sum(first))
    pool.step(first)
    t.update(act_seq_kv=got[1], free_count=got[2])
    new, tokens, code = [1] * 300, 300, 2
    if what == "negative":
        t["act_seq_kv"][77] = -1
    elif what == "table":
        new[5] = 65
        tokens = 400
    elif what == "ended_table":
        t["act_seq_kv"][7], new[7] = 65, -1
    elif what == "tokens":
        tokens = 299
    elif what == "pool":
        code = 5
        t["free_count"].fill_(3)
    elif what == "count":
        code = 5
        t["free_count"].fill_(1211)
    elif what == "count_low":
        code = 5
        t["free_count"].fill_(-1)
    elif what == "returned":
        code = 5
        new[59] = -1
        t["free_count"].fill_(1210)
    before = {k: v.clone() for k, v in t.items()}
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    q, kv, count, slots, pos = _plan(t, new, 16, tokens, error=err)
    assert err.item() == code
    assert all(torch.equal(t[k], before[k]) for k in t)
    assert not bool(q.any()) and torch.equal(kv, t["act_seq_kv"]) and torch.equal(count, t["free_count"])
    assert bool((slots == -1).all()) and bool((pos == -1).all())


@pytest.mark.gpu
@pytest.mark.parametrize("page", [-1, 12, 2 ** 31 - 1, -2 ** 31])
def test_a_page_outside_the_cache(page):
    """It gives its tokens no slot, and its request's others theirs."""
    i = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    t = dict(block_table=i([[0, 1, 2], [page, 3, 4]]), act_seq_kv=i([17, 10]), free_pages=i([5, 6, 7] + [0] * 9), free_count=i([3]))
    err = i([0])
    _, kv, count, slots, pos = _plan(t, [1, 8], 16, 9, error=err)
    assert err.item() == 3
    assert kv.tolist() == [18, 18] and count.tolist() == [2]
    assert slots.tolist() == [17] + [-1] * 6 + [7 * 16, 7 * 16 + 1]
    assert pos.tolist() == [17] + list(range(10, 18))


@pytest.mark.gpu
def test_captured_step():
    """A step captured once and replayed on lengths that the graph itself carries on."""
    pool = Pool(40, 8, 300, 16, seed=4)
    t = pool.tensors()
    new = torch.ones(40, dtype=torch.int32, device="cuda")
    out = tuple(torch.empty(n, dtype=torch.int32, device="cuda") for n in (40, 40, 1, 40, 40))
    call = lambda: sfa.page_plan(t["block_table"], t["act_seq_kv"], new, t["free_pages"], t["free_count"], page_size=16,  # noqa: E731
                                 tokens=40, outputs=out)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        assert call() is out
        t["act_seq_kv"].copy_(out[1])
        t["free_count"].copy_(out[2])
    for step in range(20):
        ended = [3, 20] if step == 9 else []
        new.fill_(1)
        for b in ended:
            new[b] = -1
        host = [-1 if b in ended else 1 for b in range(40)]
        g.replay()
        torch.cuda.synchronize()
        _same(t, out, pool.step(host), pool, 40)


def test_refusals():
    from sfa_grad_gb300.latent import PlanParams, _lib
    L, f = _lib(), ctypes.c_void_p(256)
    good = dict(B=3, max_pages=4, num_pages=12, page_size=16, tokens=5)
    for over in (dict(B=0), dict(B=8193), dict(max_pages=0), dict(max_pages=2 ** 30), dict(num_pages=0), dict(num_pages=2 ** 30),
                 dict(page_size=8), dict(page_size=24), dict(page_size=2048), dict(tokens=-1), dict(tokens=2 ** 31)):
        p = PlanParams(**{**good, **over})
        assert L.sfa_page_plan(ctypes.byref(p), *[f] * 11, None) == sfa.SFA_ERR_SHAPE, over
    p = ctypes.byref(PlanParams(**good))
    v = lambda x: ctypes.c_void_p(x)  # noqa: E731
    apart = [v(4096 * (k + 1)) for k in range(11)]
    # table, kv, new, free, count; q, kv, count, slots, positions, error: what is written overlaps nothing
    for i, k in ((5, 1), (6, 1), (7, 4), (8, 9), (5, 6), (10, 7), (9, 3), (8, 0), (0, 3), (6, 2), (10, 4), (0, 1), (3, 4)):
        a = list(apart)
        a[i] = v(a[k].value)
        assert L.sfa_page_plan(p, *a, None) == sfa.SFA_ERR_PARAM_INVALID, (i, k)
    a = list(apart)
    a[6] = v(a[1].value + 8)         # the last of three lengths
    assert L.sfa_page_plan(p, *a, None) == sfa.SFA_ERR_PARAM_INVALID
    assert L.sfa_page_plan(None, *[f] * 11, None) == sfa.SFA_ERR_NULLPTR
    for i in range(10):
        a = list(apart)
        a[i] = None
        assert L.sfa_page_plan(p, *a, None) == sfa.SFA_ERR_NULLPTR, i
    for i in range(11):
        a = list(apart)
        a[i] = v(a[i].value + 2)
        assert L.sfa_page_plan(p, *a, None) == sfa.SFA_ERR_PARAM_INVALID, i
    i = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    with pytest.raises(ValueError, match="act_seq_kv"):
        sfa.page_plan(i(3, 4), i(2), i(3), i(12), i(1), page_size=16, tokens=5)
    with pytest.raises(ValueError, match="block_table"):
        sfa.page_plan(i(3), i(3), i(3), i(12), i(1), page_size=16, tokens=5)
    with pytest.raises(ValueError, match="tokens"):
        sfa.page_plan(i(3, 4), i(3), i(3), i(12), i(1), page_size=16, tokens=-1)
    with pytest.raises(ValueError, match="outputs: slots"):
        sfa.page_plan(i(3, 4), i(3), i(3), i(12), i(1), page_size=16, tokens=5, outputs=(i(3), i(3), i(1), i(4), i(5)))
    with pytest.raises(ValueError, match="CUDA"):
        sfa.page_plan(i(3, 4), i(3), i(3), i(12), i(1), page_size=16, tokens=5)
