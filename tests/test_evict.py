"""Eviction by weight and the pages that it leaves free, against a plain
definition (sorted lists in Python); every result is exact."""
import ctypes
import math

import numpy as np
import pytest
import torch

import long_context_sparse_gb300 as dsa
from long_context_sparse_gb300 import build as dsa_build
from tests.test_serving import BF, DEV
from tests.test_tree import P, i32, refusals, scfg

gpu = pytest.mark.gpu


# ----------------------------------------------------- plain definitions


def plain_keep(w, left, n_first, n_last):
    """For each place below `left` the place whose token it holds afterwards."""
    n = len(w)
    fixed = lambda j: j < n_first or j >= n - n_last
    rank = lambda j: math.inf if fixed(j) else w[j]
    # NaN below all: its own first key
    order = sorted(range(n), key=lambda j: ((1, 0.0) if math.isnan(rank(j)) else (0, -rank(j)), j))
    kept = set(order[:left])
    freed = [j for j in range(left) if j not in kept]
    late = sorted(j for j in kept if j >= left)
    src = list(range(left))
    for a, c in zip(freed, late):
        src[a] = c
    return src


class Evict:
    def __init__(self, lens, keep, page=16, d=128, kv=1, weights="random", seed=1, extra=0):
        g = torch.Generator().manual_seed(seed)
        self.lens, self.keep, self.kv, self.page, self.d = lens, keep, kv, page, d
        need = [-(-n // page) for n in lens]
        n_pages = sum(need) + 3
        width = max([1] + need) + extra
        perm = torch.randperm(n_pages, generator=g).to(torch.int32)
        self.table = torch.full((len(lens), width), -1, dtype=torch.int32)
        at = 0
        for b, n in enumerate(need):
            self.table[b, :n] = perm[at:at + n]
            at += n
        self.cache = [torch.randn((n_pages, page, d), generator=g).to(BF) for _ in range(kv)]
        w = torch.randn((n_pages, page), generator=g)
        if weights == "few":        # many ties
            w = torch.randint(0, 3, w.shape, generator=g).float() - 1
            w[w == 0] = torch.where(torch.rand(w.shape, generator=g)[w == 0] < 0.5, 0.0, -0.0)
        elif weights == "same":
            w = torch.zeros_like(w)
        elif weights == "odd":      # everything that a float can be
            pick = torch.tensor([math.nan, math.inf, -math.inf, 0.0, -0.0, 1e-45, -1e-45, 3.4e38,
                                 -3.4e38, 1.0, 1.0000001, -math.nan])
            w = pick[torch.randint(0, len(pick), w.shape, generator=g)]
        elif weights == "close":    # keys that differ in their last bits
            w = 1.0 + torch.randint(0, 200, w.shape, generator=g).float() * 2.0 ** -23
        self.w = w
        self.cfg = dsa.ServeConfig(n_pages=n_pages, max_tokens=1, batch=len(lens),
                                   max_blocks=width, page_size=page, d_qk=d, d_v=d)

    def slots(self, b, n):
        p = torch.arange(n)
        return self.table[b][p // self.page].long() * self.page + p % self.page

    def plain(self, n_first, n_last, out, rank=None):
        cache, out = [c.clone().view(-1, self.d) for c in self.cache], out.clone().view(-1)
        w = self.w.view(-1)
        rank = (self.w if rank is None else rank).view(-1)
        for b, n in enumerate(self.lens):
            slots = self.slots(b, n)
            src = plain_keep(rank[slots].tolist(), min(n, self.keep[b]), n_first, n_last)
            to, take = slots[: len(src)], slots[src]
            out[to] = w[take]
            for x, c in zip(cache, self.cache):
                x[to] = c.view(-1, self.d)[take]
        return [c.view_as(self.cache[0]) for c in cache], out.view_as(self.w)

    def run(self, n_first=0, n_last=0, in_place=False, ws=None, keep=None, lens=None, table=None,
            rank=None):
        dv = lambda t: t.to(DEV)
        cache = [dv(c) for c in self.cache]
        w = dv(self.w)
        out = w if in_place else torch.full_like(w, 7.0)
        ws = dsa.serve_workspace(self.cfg, dsa.SERVE_WS_EVICT, DEV) if ws is None else ws
        got = dsa.evict_cache(self.cfg, w, dv(self.table if table is None else table),
                              i32(self.lens if lens is None else lens),
                              i32(self.keep if keep is None else keep), cache[0],
                              v_pages=cache[1] if self.kv == 2 else None, n_first=n_first,
                              n_last=n_last, w_out=None if in_place else out, ws=ws,
                              rank_pages=None if rank is None else dv(rank))
        torch.cuda.synchronize()
        return [c.cpu() for c in cache], got.cpu(), dsa.get_device_status(ws)


def same(a, b):
    return torch.equal(torch.nan_to_num(a, nan=1234.5), torch.nan_to_num(b, nan=1234.5)) and \
        torch.equal(torch.isnan(a), torch.isnan(b))


def check_evict(e, n_first=0, n_last=0, in_place=False, ws=None):
    cache, out, status = e.run(n_first, n_last, in_place, ws)
    assert status == 0
    ref, ref_w = e.plain(n_first, n_last, e.w if in_place else torch.full_like(e.w, 7.0))
    assert same(out, ref_w)
    for a, b in zip(cache, ref):
        assert torch.equal(a, b)


# ------------------------------------------------------------ host checks


@pytest.fixture(scope="module")
def lib():
    dsa_build.build()
    return dsa._load()


def test_evict_refusals(lib):
    c = scfg()
    r, B, slots, d = ctypes.byref(c.c()), 4, 6400, 128
    nb = dsa.serve_workspace_size(c, dsa.SERVE_WS_EVICT)
    f = lib.dsa_evict_cache
    size = dict(w=slots * 4, rank=slots * 4, table=B * 40, seq=16, keep=16, k=slots * d * 2, v=slots * d * 2,
                out=slots * 4, ws=nb)

    def call(at, first=0, last=0, ws_bytes=nb, **over):
        w, rank, table, seq, keep, k, v, out, ws = (P(x) for x in {**at, **over}.values())
        return f(r, w, rank, table, seq, keep, first, last, k, v, out, ws, ws_bytes, None)

    refusals(call, size, ("k", "v", "out", "ws"), (("out", "w"),))
    at = {n: (i + 1) << 28 for i, n in enumerate(size)}
    assert call(at, out=at["w"] + 256) == 1
    assert call(at, v=at["k"]) == 1                     # one cache twice
    assert call(at, first=-1) == 1 and call(at, last=-1) == 1
    assert call(at, keep=None) == 1 and call(at, k=None) == 1
    assert call(at, k=at["k"] + 8) == 4 and call(at, ws=at["ws"] + 16) == 4
    assert call(at, ws_bytes=nb - 1) == 3
    for over in (dict(d_qk=96, d_v=96), dict(page_size=48), dict(max_blocks=(1 << 16) + 1)):
        with pytest.raises(dsa.DsaError) as e:
            dsa.serve_workspace_size(scfg(**over), dsa.SERVE_WS_EVICT)
        assert e.value.code == 2


def test_release_refusals(lib):
    c = scfg()
    r, B, n_max = ctypes.byref(c.c()), 4, 50
    f = lib.dsa_release_pages
    size = dict(seq=16, keep=16, table=B * 40, lens=16, pages=n_max * 4, n=4, ws=256)

    def call(at, n_max=n_max, ws_bytes=256, **over):
        seq, keep, table, lens, pages, n, ws = (P(x) for x in {**at, **over}.values())
        return f(r, seq, keep, table, lens, pages, n_max, n, ws, ws_bytes, None)

    refusals(call, size, ("lens", "pages", "n", "ws"))
    at = {n: (i + 1) << 28 for i, n in enumerate(size)}
    assert call(at, pages=None) == 1 and call(at, n_max=-1) == 1 and call(at, n=None) == 1
    assert call(at, pages=at["pages"] + 2) == 4 and call(at, lens=at["lens"] + 4) == 4
    assert call(at, ws_bytes=255) == 3


def test_python_refuses_wrong_evict_tensors():
    with pytest.raises(ValueError):
        dsa.evict_cache(scfg(), torch.zeros(100, 64), None, None, None, None)
    with pytest.raises(ValueError):
        dsa.release_pages(scfg(), torch.zeros(4, dtype=torch.int32), None, None)


def test_the_plain_choice():
    assert plain_keep([5.0, 1.0, 4.0, 3.0], 2, 0, 0) == [0, 2]
    assert plain_keep([0.0, 0.0, 0.0], 2, 0, 0) == [0, 1]
    assert plain_keep([0.0, 9.0, math.nan, 1.0], 2, 1, 1) == [0, 3]
    assert plain_keep([1.0, 2.0], 0, 0, 0) == []
    assert plain_keep([math.nan, -math.inf], 1, 0, 0) == [1]


# -------------------------------------------------------------- eviction


@gpu
@pytest.mark.parametrize("weights", ["random", "few", "same", "odd", "close"])
@pytest.mark.parametrize("page,d,kv", [(16, 128, 1), (64, 512, 2), (128, 256, 1)])
def test_evict(weights, page, d, kv):
    lens = [0, 1, 2, 15, 16, 17, 31, 32, 33, 100, 300, 511, 513, 1000]
    keep = [0, 0, 1, 15, 9, 17, 1, 31, 16, 64, 299, 0, 512, 500]
    e = Evict(lens, keep, page, d, kv, weights, seed=page)
    check_evict(e)
    check_evict(e, n_first=4, n_last=10)
    check_evict(e, n_first=3, n_last=5, in_place=True)


@gpu
@pytest.mark.parametrize("n,keep,extra", [
    (4000, 2000, 0), (5000, 100, 0), (9000, 4500, 0), (20000, 19999, 0), (70000, 20000, 0),
    (300, 150, 2000),             # a short request where long ones are allowed
    (200, 100, 26000)])           # and where a share would not fit shared memory
@pytest.mark.parametrize("weights", ["random", "few", "odd"])
def test_evict_long(n, keep, extra, weights):
    e = Evict([n, n // 2, 7], [keep, n // 3, 9], 16, 128, 2, weights, seed=n, extra=extra)
    check_evict(e, n_first=1, n_last=n // 10)


@gpu
def test_evict_past_shared_memory():
    """More tokens than the keys of eight CTAs hold."""
    e = Evict([410000], [100000], 128, 128, 1, "random", seed=3)
    check_evict(e, n_last=1000)
    e.w = torch.zeros_like(e.w)
    check_evict(e, n_first=5, n_last=1000, in_place=True)


@gpu
@pytest.mark.parametrize("weights", ["random", "few"])
def test_evict_more_than_the_gpu_has_room_for(weights):
    """Many requests, some of whose shares pass shared memory while others' do not: a CTA
    each, and clusters as the longest cache that is allowed wants them."""
    check_evict(Evict([60000, 100, 0, 40000] + [50] * 77, [30000, 60, 5, 39000] + [20] * 77, 16,
                      128, 1, weights, seed=11), n_first=1, n_last=40)
    check_evict(Evict([300000, 100000, 7] + [40] * 97, [1000, 50000, 3] + [30] * 97, 128, 128, 1,
                      weights, seed=12, extra=(1 << 15) - 2344), n_last=9, in_place=True)


@gpu
@pytest.mark.parametrize("in_place", [False, True])
def test_ranks_of_their_own(in_place):
    """Rejected drafts: -inf among +inf; and any ranks, the weights only carried."""
    g = torch.Generator().manual_seed(1)
    for n in (300, 6000):
        e = Evict([n, n // 3, 40], [n - 20, n // 3 - 5, 10], 16, 128, 2, "odd", seed=n)
        drafts = torch.full_like(e.w, math.inf)
        for b, m in enumerate(e.lens):
            s = e.slots(b, m)
            gone = m - 40 + torch.randperm(40, generator=g)[: m - e.keep[b]]
            drafts.view(-1)[s[gone]] = -math.inf
        for rank in (drafts, torch.randn(e.w.shape, generator=g)):
            cache, out, status = e.run(in_place=in_place, rank=rank)
            ref, ref_w = e.plain(0, 0, e.w if in_place else torch.full_like(e.w, 7.0), rank)
            assert status == 0 and same(out, ref_w)
            for a, b in zip(cache, ref):
                assert torch.equal(a, b)


@gpu
def test_more_protected_than_the_budget():
    e = Evict([100, 60], [30, 50], 16, 128, 1, "random", seed=4)
    check_evict(e, n_first=20, n_last=80)
    check_evict(e, n_first=1 << 40, n_last=1 << 40)
    check_evict(e, n_first=0, n_last=1 << 31)


@gpu
def test_many_requests_twice_with_one_workspace():
    rng = np.random.default_rng(5)
    lens = rng.integers(0, 200, 1500).tolist()
    keep = rng.integers(0, 150, 1500).tolist()
    e = Evict(lens, keep, 16, 128, 1, "few", seed=5)
    ws = dsa.serve_workspace(e.cfg, dsa.SERVE_WS_EVICT, DEV)
    for _ in range(3):              # the counters are left as they were found
        check_evict(e, n_first=2, ws=ws)
    ws2 = torch.randint(0, 255, ws.shape, dtype=torch.uint8, device=DEV)  # only the header counts
    ws2[:256] = 0
    check_evict(e, n_first=2, ws=ws2)


@gpu
def test_evict_latches_and_leaves_bad_requests():
    e = Evict([100, 50, 80], [40, 20, 30], 16, 128, 1, "random", seed=6)
    for lens, keep in (([100, 9999, 80], None), ([100, -1, 80], None), (None, [40, -1, 30])):
        cache, out, status = e.run(lens=lens, keep=keep)
        assert status == 7
        ref, ref_w = e.plain(0, 0, torch.full_like(e.w, 7.0))
        mine = e.slots(1, 50)
        assert torch.equal(cache[0].view(-1, 128)[mine], e.cache[0].view(-1, 128)[mine])
        assert (out.view(-1)[mine] == 7.0).all()
        for b, n in ((0, 100), (2, 80)):
            s = e.slots(b, n)
            assert torch.equal(cache[0].view(-1, 128)[s], ref[0].view(-1, 128)[s])
            assert same(out.view(-1)[s], ref_w.view(-1)[s])
    t = e.table.clone()
    t[0, 1], t[2, 0] = 12345, -9
    cache, out, status = e.run(table=t)
    assert status == 7
    s = e.slots(1, 50)
    ref, ref_w = e.plain(0, 0, torch.full_like(e.w, 7.0))
    assert torch.equal(cache[0].view(-1, 128)[s], ref[0].view(-1, 128)[s])


@gpu
def test_a_page_that_stands_in_many_places_stays_in_bounds():
    """More moves than the cache has slots for: latched, nothing out of bounds."""
    e = Evict([64] * 200, [32] * 200, 16, 128, 1, "random", seed=8)
    e2 = Evict([64], [32], 16, 128, 1, "random", seed=8)
    e2.cfg = dsa.ServeConfig(n_pages=e2.cache[0].shape[0], max_tokens=1, batch=200, max_blocks=4,
                             page_size=16, d_qk=128, d_v=128)
    e2.lens, e2.keep = e.lens, e.keep
    table = e2.table[:1, :4].repeat(200, 1)
    table = table[:, torch.tensor([0, 1, 2, 3])].contiguous()
    need = dsa.serve_workspace_size(e2.cfg, dsa.SERVE_WS_EVICT)
    ws = torch.zeros(need + 4096, dtype=torch.uint8, device=DEV)
    ws[256:] = 255
    guard = ws[need:].clone()
    _, _, status = e2.run(ws=ws, table=table)
    assert status == 7 and torch.equal(ws[need:], guard)


# --------------------------------------------------------------- release


@gpu
@pytest.mark.parametrize("B,page,hi", [(1, 16, 50), (5, 64, 300), (256, 16, 100), (257, 32, 900),
                                       (3000, 128, 2000)])
def test_release(B, page, hi):
    rng = np.random.default_rng(B)
    lens, keep = rng.integers(0, hi, B).tolist(), rng.integers(0, hi, B).tolist()
    width = -(-hi // page)
    table = rng.integers(0, 1000, (B, width)).astype(np.int32)
    cfg = scfg(n_pages=1 << 20, batch=B, max_blocks=width, page_size=page)
    left = [min(a, b) for a, b in zip(lens, keep)]
    pages = [p for b in range(B)
             for p in table[b, -(-left[b] // page): -(-lens[b] // page)].tolist()]
    ws = dsa.serve_workspace(cfg, dsa.SERVE_WS_TABLES, DEV)
    r = dsa.release_pages(cfg, i32(lens), i32(keep), torch.from_numpy(table).to(DEV), ws=ws)
    assert dsa.get_device_status(ws) == 0
    assert r.new_lens.tolist() == left and r.n_released.item() == len(pages)
    assert r.pages[: len(pages)].tolist() == pages and (r.pages[len(pages):] == -1).all()
    if len(pages) > 2:              # a list that is too short, at an odd place
        n = len(pages) // 2
        big = torch.full((n + 2,), -5, dtype=torch.int32, device=DEV)
        out = dsa.ReleasedPages(torch.empty_like(r.new_lens), big[1:n + 1],
                                torch.empty_like(r.n_released))
        dsa.release_pages(cfg, i32(lens), i32(keep), torch.from_numpy(table).to(DEV), out=out,
                          ws=ws)
        assert dsa.get_device_status(ws) == 10
        assert big.tolist() == [-5] + pages[:n] + [-5]
        assert out.n_released.item() == len(pages)


@gpu
def test_release_latches_bad_lengths():
    cfg = scfg(batch=4, max_blocks=4, page_size=16)
    table = torch.arange(16, dtype=torch.int32, device=DEV).view(4, 4)
    ws = dsa.serve_workspace(cfg, dsa.SERVE_WS_TABLES, DEV)
    r = dsa.release_pages(cfg, i32([65, 64, -3, 40]), i32([1, 1, 1, -1]), table, ws=ws)
    assert dsa.get_device_status(ws) == 7
    assert r.new_lens.tolist() == [65, 1, -3, 40]
    assert r.n_released.item() == 3 and r.pages[:3].tolist() == [5, 6, 7]
