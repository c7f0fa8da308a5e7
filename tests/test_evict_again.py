"""Evictions one after the other, and of requests that have pages outside the cache: what
an earlier call or another request leaves behind does not reach a request."""
import math

import pytest
import torch

import long_context_sparse_gb300 as dsa
from tests.test_evict import Evict, plain_keep, same
from tests.test_serving import DEV
from tests.test_tree import i32

gpu = pytest.mark.gpu


@gpu
def test_moves_of_an_earlier_call_are_not_made_again():
    """A list full of moves, then a call whose requests share a page: some of them find no
    place in the list, and what stands there instead is an earlier call's."""
    e = Evict([640], [320], 16, 128, 2, "random", seed=21)
    n_pages = e.cache[0].shape[0]
    cfg = dsa.ServeConfig(n_pages=n_pages, max_tokens=1, batch=16, max_blocks=40, page_size=16,
                          d_qk=128, d_v=128)
    table = e.table.repeat(16, 1)
    ws = dsa.serve_workspace(cfg, dsa.SERVE_WS_EVICT, DEV)
    cache = [c.to(DEV) for c in e.cache]
    w = e.w.to(DEV)

    def evict(lens, keep, out):
        dsa.evict_cache(cfg, w, table.to(DEV), i32(lens), i32(keep), cache[0], v_pages=cache[1],
                        n_last=max(keep), w_out=out, ws=ws)
        return dsa.get_device_status(ws)

    assert evict([640] + [0] * 15, [320] + [0] * 15, torch.zeros_like(w)) == 0
    before = [c.clone() for c in cache]
    out = torch.full_like(w, 7.0)
    assert evict([100] * 16, [50] * 16, out) == 7       # 16 times 50 moves of 100 slots
    assert all(torch.equal(a, b) for a, b in zip(cache, before))
    named = torch.zeros(n_pages, dtype=torch.bool)
    named[table[0, :7].long()] = True
    assert (out[~named.to(DEV)] == 7.0).all()
    # the counters are as they were: the next call is a first one
    e.cache, e.w = [c.cpu() for c in cache], w.cpu()
    e.lens, e.keep, e.cfg = [640] + [0] * 15, [300] + [0] * 15, cfg
    e.table = table
    assert evict(e.lens, e.keep, out) == 0
    ref, _ = e.plain(0, 300, e.w)
    for a, b in zip(cache, ref):
        assert torch.equal(a.cpu(), b)


def plain_keep_bad(w, bad, left, n_first, n_last):
    """plain_keep where bad[j]: place j lies on a page outside the cache."""
    n = len(w)

    def order(j):
        if bad[j]:
            return 2, 0.0, j
        rank = math.inf if j < n_first or j >= n - n_last else w[j]
        return (1, 0.0, j) if math.isnan(rank) else (0, -rank, j)

    kept = set(sorted(range(n), key=order)[:left])
    freed = [j for j in range(left) if j not in kept]
    src = list(range(left))
    for a, c in zip(freed, sorted(j for j in kept if j >= left)):
        src[a] = c
    return src


def test_the_plain_choice_with_bad_pages():
    none = [False] * 4
    for w, first, last in (([0.0, 9.0, math.nan, 1.0], 1, 1), ([1.0, 1.0, 2.0, 0.0], 0, 0)):
        for left in range(5):
            assert plain_keep_bad(w, none, left, first, last) == plain_keep(w, left, first, last)
    nan = math.nan
    assert plain_keep_bad([5.0, nan, 1.0], [True, False, False], 2, 3, 0) == [2, 1]
    assert plain_keep_bad([5.0, nan, 1.0], [True, False, False], 1, 0, 0) == [2]


def check_bad_pages(e, table, n_first, n_last):
    """Every row of every request, and all that belongs to none, against the definition."""
    cache, out, status = e.run(n_first, n_last, table=table)
    assert status == 7
    ref, want = [c.view(-1, e.d).clone() for c in e.cache], torch.full_like(e.w, 7.0).view(-1)
    for b, n in enumerate(e.lens):
        p = torch.arange(n)
        page = table[b][p // e.page].long()
        bad = (page < 0) | (page >= e.w.shape[0])
        slots = torch.where(bad, 0, page) * e.page + p % e.page
        w = torch.where(bad, 0.0, e.w.view(-1)[slots]).tolist()
        src = plain_keep_bad(w, bad.tolist(), min(n, e.keep[b]), n_first, n_last)
        for to, at in enumerate(src):
            if bad[to] or bad[at]:
                continue
            want[slots[to]] = e.w.view(-1)[slots[at]]
            for x, c in zip(ref, e.cache):
                x[slots[to]] = c.view(-1, e.d)[slots[at]]
    assert same(out.view(-1), want)
    for x, y in zip(cache, ref):
        assert torch.equal(x.view(-1, e.d), y)


def with_bad_pages(e, seed):
    g = torch.Generator().manual_seed(seed)
    n_pages = e.cache[0].shape[0]
    odd = torch.tensor([-1, -9, n_pages, 1 << 30, -(1 << 31)], dtype=torch.int32)
    t = e.table.clone()
    for b, n in enumerate(e.lens):
        for i in range(-(-n // e.page)):
            if torch.rand((), generator=g) < (0.0, 0.1, 0.5, 0.95, 1.0)[b % 5]:
                t[b, i] = odd[torch.randint(0, 5, (), generator=g)]
    return t


@gpu
@pytest.mark.parametrize("weights", ["random", "few", "odd"])
@pytest.mark.parametrize("lens,keep,extra", [
    ([100, 300, 64, 200, 90, 17, 33, 500, 400, 90], [40, 200, 30, 150, 50, 9, 33, 250, 399, 1], 0),
    ([9000, 8000, 700, 5000, 100], [4000, 7000, 300, 2500, 40], 0),   # clusters
    ([300, 500, 200, 100, 64], [100, 400, 90, 70, 30], 26000)])       # keys not in shared memory
def test_requests_with_bad_pages(weights, lens, keep, extra):
    e = Evict(lens, keep, 16, 128, 2, weights, seed=len(lens), extra=extra)
    for n_first, n_last in ((0, 0), (5, 60)):
        check_bad_pages(e, with_bad_pages(e, n_last), n_first, n_last)


@gpu
def test_bad_pages_leave_the_others_their_moves():
    """Requests that have no page at all, and would move far more tokens than the cache
    holds; some of whose protected tokens stand on pages of theirs."""
    e = Evict([60, 600] + [640] * 14, [30, 300] + [320] * 14, 16, 128, 1, "random", seed=31)
    n_pages = 4 + 38 + 2
    t = torch.full((16, 40), -1, dtype=torch.int32)
    perm = torch.randperm(n_pages, generator=torch.Generator().manual_seed(1)).to(torch.int32)
    t[0, :4], t[1, :38] = perm[:4], perm[4:42]
    t[2, 39] = perm[42]
    e.cache, e.w = [c[:n_pages].contiguous() for c in e.cache], e.w[:n_pages].contiguous()
    e.cfg = dsa.ServeConfig(n_pages=n_pages, max_tokens=1, batch=16, max_blocks=40, page_size=16,
                            d_qk=128, d_v=128)
    for n_last in (0, 30, 320):
        check_bad_pages(e, t, 0, n_last)


@gpu
def test_more_long_requests_than_sms():
    """A CTA a request, whose keys take more than half of an SM's shared memory."""
    lens = [22000 + 97 * b % 9000 for b in range(160)]
    e = Evict(lens, [n // 3 if b % 3 else n - 5 for b, n in enumerate(lens)], 128, 128, 1, "few",
              seed=41)
    cache, out, status = e.run(3, 50)
    assert status == 0
    for b in range(0, 160, 13):
        s = e.slots(b, lens[b])
        src = plain_keep(e.w.view(-1)[s].tolist(), e.keep[b], 3, 50)
        assert same(out.view(-1)[s[: len(src)]], e.w.view(-1)[s[src]])
        assert torch.equal(cache[0].view(-1, 128)[s[: len(src)]],
                           e.cache[0].view(-1, 128)[s[src]])
