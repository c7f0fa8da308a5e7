"""Eviction that knows the tokens' ages, against a plain definition, and as a serving
loop has it: a few new tokens, then back to the budget, step after step."""
import ctypes
import math

import pytest
import torch

import long_context_sparse_gb300 as dsa
from long_context_sparse_gb300 import build as dsa_build
from tests.test_evict import Evict, plain_keep, same
from tests.test_serving import BF, DEV
from tests.test_serving_early import late, replayed  # noqa: F401 (a fixture)
from tests.test_tree import P, i32, refusals, scfg

gpu = pytest.mark.gpu
LO, HI = -(1 << 31), (1 << 31) - 1


def plain_keep_aged(w, pos, next_pos, left, n_first, n_last):
    """plain_keep where the protected tokens are those of the first and last positions."""
    fixed = [p < n_first or p >= next_pos - n_last for p in pos]
    return plain_keep([math.inf if f else x for f, x in zip(fixed, w)], left, 0, 0)


def test_the_plain_choice_by_age():
    w = [5.0, 1.0, 2.0, 3.0, 0.0]
    for first in range(3):
        for last in range(3):       # in order of time: as by place
            for left in range(6):
                assert plain_keep_aged(w, range(5), 5, left, first, last) == \
                    plain_keep(w, left, first, last)
    assert plain_keep_aged(w, [0, 4, 2, 3, 1], 5, 2, 1, 1) == [0, 1]


# ------------------------------------------------------------ host checks


@pytest.fixture(scope="module")
def lib():
    dsa_build.build()
    return dsa._load()


def test_aged_refusals(lib):
    c = scfg()
    r, B, slots, d = ctypes.byref(c.c()), 4, 6400, 128
    nb = dsa.serve_workspace_size(c, dsa.SERVE_WS_EVICT)
    f = lib.dsa_evict_cache_aged
    size = dict(w=slots * 4, rank=slots * 4, pos=slots * 4, next=16, table=B * 40, seq=16, keep=16,
                k=slots * d * 2, v=slots * d * 2, out=slots * 4, ws=nb)

    def call(at, first=0, last=0, ws_bytes=nb, **over):
        w, rank, pos, nxt, table, seq, keep, k, v, out, ws = (P(x) for x in
                                                              {**at, **over}.values())
        return f(r, w, rank, pos, nxt, table, seq, keep, first, last, k, v, out, ws, ws_bytes, None)

    refusals(call, size, ("pos", "k", "v", "out", "ws"), (("out", "w"),))
    at = {n: (i + 1) << 28 for i, n in enumerate(size)}
    assert call(at, pos=None) == 1 and call(at, next=None) == 1
    assert call(at, pos=at["pos"] + 4) == 4 and call(at, next=at["next"] + 4) == 4
    assert call(at, first=-1) == 1 and call(at, last=-1) == 1


def test_python_wants_positions_and_the_next_ones():
    with pytest.raises(ValueError):
        dsa.evict_cache(scfg(), torch.zeros(100, 64), None, None, None, None, pos_pages=None,
                        next_pos=torch.zeros(4))


# ------------------------------------------------------ against the definition


def run(e, pos, nxt, n_first, n_last, in_place=False, ws=None, rank=None):
    dv = lambda t: t.to(DEV)
    cache, w, pos = [dv(c) for c in e.cache], dv(e.w), dv(pos)
    out = w if in_place else torch.full_like(w, 7.0)
    ws = dsa.serve_workspace(e.cfg, dsa.SERVE_WS_EVICT, DEV) if ws is None else ws
    got = dsa.evict_cache(e.cfg, w, dv(e.table), i32(e.lens), i32(e.keep), cache[0],
                          v_pages=cache[1] if e.kv == 2 else None, n_first=n_first, n_last=n_last,
                          w_out=None if in_place else out, ws=ws,
                          rank_pages=None if rank is None else dv(rank), pos_pages=pos,
                          next_pos=i32(nxt))
    assert dsa.get_device_status(ws) == 0
    return [c.cpu() for c in cache], got.cpu(), pos.cpu()


def check_aged(e, pos, nxt, n_first, n_last, in_place=False, rank=None):
    cache, out, got = run(e, pos, nxt, n_first, n_last, in_place, rank=rank)
    ref = [c.clone().view(-1, e.d) for c in e.cache]
    want = (e.w if in_place else torch.full_like(e.w, 7.0)).clone().view(-1)
    want_pos, by = pos.clone().view(-1), (e.w if rank is None else rank).view(-1)
    for b, n in enumerate(e.lens):
        s = e.slots(b, n)
        src = plain_keep_aged(by[s].tolist(), pos.view(-1)[s].tolist(), nxt[b],
                              min(n, e.keep[b]), n_first, n_last)
        to, at = s[: len(src)], s[src]
        want[to], want_pos[to] = e.w.view(-1)[at], pos.view(-1)[at]
        for x, c in zip(ref, e.cache):
            x[to] = c.view(-1, e.d)[at]
    assert same(out.view(-1), want) and torch.equal(got.view(-1), want_pos)
    for x, y in zip(cache, ref):
        assert torch.equal(x.view(-1, e.d), y)


def ages(e, seed, gaps=2):
    """Distinct positions in any order, of which some tokens are gone; the next ones."""
    g = torch.Generator().manual_seed(seed)
    pos = torch.full(e.w.shape, -77, dtype=torch.int32)
    for b, n in enumerate(e.lens):
        pos.view(-1)[e.slots(b, n)] = torch.randperm(gaps * n, generator=g)[:n].to(torch.int32)
    return pos, [gaps * n for n in e.lens]


@gpu
@pytest.mark.parametrize("weights", ["random", "few", "odd"])
@pytest.mark.parametrize("page,d,kv", [(16, 128, 1), (64, 512, 2), (128, 256, 1)])
def test_evict_by_age(weights, page, d, kv):
    lens = [0, 1, 2, 15, 16, 17, 31, 32, 33, 100, 300, 511, 513, 1000]
    keep = [0, 0, 1, 15, 9, 17, 1, 31, 16, 64, 299, 0, 512, 500]
    e = Evict(lens, keep, page, d, kv, weights, seed=page)
    pos, nxt = ages(e, page)
    check_aged(e, pos, nxt, 0, 0)
    check_aged(e, pos, nxt, 4, 40)
    check_aged(e, pos, nxt, 3, 25, in_place=True)
    rank = torch.randn(e.w.shape, generator=torch.Generator().manual_seed(page))
    check_aged(e, pos, nxt, 7, 80, rank=rank)


@gpu
@pytest.mark.parametrize("n,keep,extra", [(5000, 100, 0), (9000, 4500, 0), (70000, 20000, 0),
                                          (300, 150, 2000), (200, 100, 26000)])
def test_evict_by_age_long(n, keep, extra):
    e = Evict([n, n // 2, 7], [keep, n // 3, 9], 16, 128, 2, "few", seed=n, extra=extra)
    pos, nxt = ages(e, n, 3)
    check_aged(e, pos, nxt, 5, n // 4)


@gpu
def test_positions_of_all_sizes():
    """The ends of 32 bits, and more protected than there are."""
    e = Evict([100, 60], [30, 50], 16, 128, 1, "random", seed=4)
    g = torch.Generator().manual_seed(4)
    odd = torch.tensor([LO, LO + 1, -5, -1, 0, 1, 7, HI - 1, HI], dtype=torch.int64)
    pos = odd[torch.randint(0, 9, e.w.shape, generator=g)].to(torch.int32)
    for nxt in ([LO, HI], [HI, 0], [8, -4]):
        for first, last in ((0, 0), (1, 9), (HI, 0), (1 << 31, 0), (0, HI), (0, 1 << 31),
                            (0, 1 << 32), (1 << 40, 1 << 62)):
            check_aged(e, pos, nxt, first, last)


@gpu
def test_evict_by_place_leaves_no_positions_behind():
    """The same workspace for both kinds of call, in turns."""
    e = Evict([300, 90, 2000], [120, 50, 900], 16, 128, 1, "random", seed=6)
    pos, nxt = ages(e, 6)
    ws = dsa.serve_workspace(e.cfg, dsa.SERVE_WS_EVICT, DEV)
    want = run(e, pos, nxt, 2, 100)
    by_place = e.run(2, 100)
    for _ in range(3):
        for a, b in zip(run(e, pos, nxt, 2, 100, ws=ws), want):
            assert all(same(x, y) for x, y in zip(a, b)) if isinstance(a, list) else same(a, b)
        got = e.run(2, 100, ws=ws)
        assert same(got[1], by_place[1]) and torch.equal(got[0][0], by_place[0][0])


# ---------------------------------------------------------- a serving loop


@gpu
@pytest.mark.parametrize("aged", [True, False])
@pytest.mark.parametrize("new", [1, 4, 16])
def test_the_newest_tokens_stay(new, aged):
    """Steps of `new` tokens a request, each followed by an eviction to the budget: the first
    4 and the last 64 tokens are there after every step, however little weight they have.
    By place the newest ones are lost, which is why there is the other."""
    B, d, page, budget, first, last, steps = 3, 128, 16, 100, 4, 64, 400 // new
    width = (budget + new + page - 1) // page
    n_pages, T = B * width + 1, B * new
    cfg = dsa.ServeConfig(n_pages=n_pages, max_tokens=T, batch=B, max_blocks=width, page_size=page,
                          d_qk=d, d_v=d)
    g = torch.Generator().manual_seed(new)
    # a slot more than the cache has: where rows of no request (slot -1) enter their position
    flat = torch.zeros(n_pages * page + 1, dtype=torch.int32, device=DEV)
    pos = flat[:-1].view(n_pages, page)
    k = torch.zeros((n_pages, page, d), dtype=BF, device=DEV)
    w = torch.zeros((n_pages, page), device=DEV)
    table = torch.full((B, width), -1, dtype=torch.int32, device=DEV)
    ws = {x: dsa.serve_workspace(cfg, x, DEV) for x in (dsa.SERVE_WS_TABLES, dsa.SERVE_WS_APPEND,
                                                        dsa.SERVE_WS_EVICT)}
    free, lens = list(range(n_pages)), [0] * B
    forgotten = 0
    for step in range(steps):
        t = dsa.build_page_tables(cfg, i32(lens), i32([new] * B), i32(free), table,
                                  ws=ws[dsa.SERVE_WS_TABLES])
        free = free[t.pages_taken.item():]
        at = step * new + torch.arange(T) % new            # the rows' positions
        rows = torch.zeros((T, d))
        rows[:, 0], rows[:, 1], rows[:, 2] = at // 128, at % 128, torch.arange(T) // new
        dsa.append_cache(cfg, t.slot_map, rows.to(BF).to(DEV), k, ws=ws[dsa.SERVE_WS_APPEND])
        slots = t.slot_map.long()
        flat[slots] = at.to(torch.int32).to(DEV)
        w.view(-1)[slots] = torch.rand(T, generator=g).to(DEV) * 1e-3 - 1.0
        seq, keep, nxt = t.seq_lens, i32([budget] * B), i32([(step + 1) * new] * B)
        old = seq.tolist()
        dsa.evict_cache(cfg, w, table, seq, keep, k, n_first=first, n_last=last,
                        ws=ws[dsa.SERVE_WS_EVICT], **(dict(pos_pages=pos, next_pos=nxt) if aged
                                                      else {}))
        r = dsa.release_pages(cfg, seq, keep, table, ws=ws[dsa.SERVE_WS_TABLES])
        free += r.pages[: r.n_released.item()].tolist()
        lens = r.new_lens.tolist()
        assert lens == [min(n, budget) for n in old]
        end, tab = (step + 1) * new, table.cpu()
        must = set(range(min(first, end))) | set(range(max(0, end - last), end))
        for b in range(B):
            j = torch.arange(lens[b])
            s = tab[b][j // page].long() * page + j % page
            held = k.cpu().view(-1, d)[s].float()
            ids = (held[:, 0] * 128 + held[:, 1]).long().tolist()
            assert (held[:, 2] == b).all() and len(set(ids)) == lens[b]
            if aged:
                assert must <= set(ids)
                assert pos.cpu().view(-1)[s].tolist() == ids
            forgotten += len(must - set(ids))
    assert all(dsa.get_device_status(x) == 0 for x in ws.values())
    assert (forgotten == 0) == aged


@gpu
@pytest.mark.parametrize("captured", [False, True])
def test_positions_that_are_written_late(late, captured):  # noqa: F811
    e = Evict([5000, 300, 20], [1000, 200, 30], 16, 128, 1, "few", seed=7)
    first, nxt = ages(e, 7)
    dv = lambda t: t.to(DEV)
    w, table, seq, keep = dv(e.w), dv(e.table), i32(e.lens), i32(e.keep)
    k0, first = dv(e.cache[0]), dv(first)
    cache, nxt = k0.clone(), i32(nxt)
    pos, out = torch.zeros(e.w.shape, dtype=torch.int32, device=DEV), torch.zeros_like(w)
    ws = dsa.serve_workspace(e.cfg, dsa.SERVE_WS_EVICT, DEV)

    def step():
        cache.copy_(k0), pos.zero_(), out.zero_()
        late(pos, first)
        dsa.evict_cache(e.cfg, w, table, seq, keep, cache, w_out=out, ws=ws, n_first=3, n_last=500,
                        pos_pages=pos, next_pos=nxt)

    pos.copy_(first)
    want_k, want_out = k0.clone(), torch.zeros_like(w)
    dsa.evict_cache(e.cfg, w, table, seq, keep, want_k, w_out=want_out, n_first=3, n_last=500,
                    pos_pages=pos, next_pos=nxt)
    want_pos = pos.clone()
    replayed(step, captured)
    torch.cuda.synchronize()
    assert torch.equal(cache, want_k) and torch.equal(out, want_out) and torch.equal(pos, want_pos)
    assert dsa.get_device_status(ws) == 0
