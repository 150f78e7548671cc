"""Plans whose pages far outnumber their tokens, and steps that do not fit while many blocks look at them."""
import random

import pytest
import torch

from test_page_plan import Pool, _plan, _same
from timing_util import in_turns


def _long(pool, lens):
    """Requests of these lengths, without going through the steps that made them."""
    for b, n in enumerate(lens):
        pool.kv[b] = n
        for j in range(pool.held(n)):
            pool.table[b][j] = pool.free.pop()
    return pool.tensors()


@pytest.mark.gpu
@pytest.mark.parametrize("room", [0, 70001])
@pytest.mark.parametrize("kinds", ["half", "all", "grow"])
def test_many_pages_and_few_tokens(kinds, room):
    """Half of the requests end, or all, or all of them begin a page with their one token."""
    batch, page, per = 700, 16, 130
    rng = random.Random(batch)
    pool = Pool(batch, per, batch * per, page, seed=3)
    lens = [16 * rng.randint(50, 129) if kinds == "grow" else rng.randint(800, 16 * 129) for _ in range(batch)]
    t = _long(pool, lens)
    new = [1 if kinds == "grow" or (kinds == "half" and b % 2) else -1 for b in range(batch)]
    tokens = sum(max(n, 0) for n in new) + room
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = _plan(t, new, page, tokens, error=err)
    _same(t, got, pool.step(new), pool, tokens)
    assert err.item() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("ended", [512, 1024])
def test_time_follows_the_pages_too(ended):
    """Some 390,000 or 790,000 pages come back, with 512 new tokens or none: as fast as with room for many
    tokens, which brings blocks of its own (one block took 496 and 981 us, with room 10 and 11)."""
    import sfa_grad_gb300 as sfa
    batch, page, per = 1024, 16, 1025
    rng = random.Random(2)
    pool = Pool(batch, per, batch * per, page)
    t = _long(pool, [rng.randint(8192, 16384) for _ in range(batch)])
    new = torch.tensor([-1 if ended == batch or b % 2 else 1 for b in range(batch)], dtype=torch.int32, device="cuda")
    calls = []
    for tokens in (int((new > 0).sum()), 152 * 512):
        out = tuple(torch.empty(n, dtype=torch.int32, device="cuda") for n in (batch, batch, 1, tokens, tokens))
        calls.append(lambda out=out, tokens=tokens: sfa.page_plan(
            t["block_table"], t["act_seq_kv"], new, t["free_pages"], t["free_count"], page_size=page, tokens=tokens,
            outputs=out))
    few, many = in_turns(*calls, each=5)
    assert few <= 3 * many, (few, many)


@pytest.mark.gpu
@pytest.mark.parametrize("what", ["negative", "table", "tokens", "pool", "count", "returned"])
def test_many_blocks_change_nothing(what):
    """Room for 40,000 tokens, and 700 requests of many pages: every block finds that the step does not fit."""
    batch, page, per, room = 700, 16, 64, 40000
    rng = random.Random(5)
    pool = Pool(batch, per, batch * per, page, seed=9)
    t = _long(pool, [rng.randint(1, 1000) for _ in range(batch)])
    new, code = [(-1, 1, 0)[b % 3] for b in range(batch)], 2
    if what == "negative":
        t["act_seq_kv"][699] = -1
    elif what == "table":
        t["act_seq_kv"][600], new[600] = 1000, 25
    elif what == "tokens":
        new = [58] * batch
        t["act_seq_kv"].clamp_(max=900)
    elif what == "pool":
        code, new = 5, [17] * batch
        t["act_seq_kv"].clamp_(max=900)
        t["free_count"].fill_(11)
    elif what == "count":
        code = 5
        t["free_count"].fill_(batch * per + 1)
    elif what == "returned":
        code = 5
        t["free_count"].fill_(batch * per)
    before = {k: v.clone() for k, v in t.items()}
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    q, kv, count, slots, pos = _plan(t, new, page, room, error=err)
    assert err.item() == code
    assert all(torch.equal(t[k], before[k]) for k in t)
    assert not bool(q.any()) and torch.equal(kv, t["act_seq_kv"]) and torch.equal(count, t["free_count"])
    assert bool((slots == -1).all()) and bool((pos == -1).all())


@pytest.mark.gpu
def test_a_length_lowered_between_steps():
    """Tokens of a draft taken back: within the last page nothing else changes; past its border the caller
    returns the pages behind, and no page is lost or held twice."""
    page, batch = 16, 3
    pool = Pool(batch, 8, 12, page, seed=1)
    t = pool.tensors()
    for new, taken in (([20, 30, 5], [0, 0, 0]), ([6, 5, 9], [3, 2, 0]), ([7, 1, 9], [6, 0, 4]), ([40, -1, 1], [38, 0, 0]),
                       ([1, 60, 3], [0, 59, 3]), ([-1, -1, -1], [0, 0, 0])):
        tokens = sum(max(n, 0) for n in new)
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        got = _plan(t, new, page, tokens, error=err)
        _same(t, got, pool.step(new), pool, tokens)
        assert err.item() == 0
        for b, n in enumerate(taken):
            left = pool.kv[b] - n
            pool.free += pool.table[b][pool.held(left):pool.held(pool.kv[b])]
            pool.kv[b] = left
        held = [p for b in range(batch) for p in pool.table[b][:pool.held(pool.kv[b])]]
        assert sorted(held + pool.free) == list(range(12))
        t = pool.tensors()
    assert pool.kv == [0, 0, 0] and len(pool.free) == 12
