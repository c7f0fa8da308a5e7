"""The serving calls: page tables, cache append and shared-prefix attention,
against plain definitions (integers in Python, attention in fp64)."""
import copy
import ctypes
import dataclasses
import json
import math
import os
import pickle
import subprocess
import sys

import numpy as np
import pytest
import torch

import long_context_sparse_gb300 as dsa
from long_context_sparse_gb300 import build as dsa_build

gpu = pytest.mark.gpu
DEV = torch.device("cuda", 0)
BF = torch.bfloat16

# Tolerances, from the roundings on the way (bf16: 2^-8 relative).  O: one
# rounding of each P to bf16 as a tensor-core operand (2^-8 sum_j P_j |v_j|;
# the row sum is taken of the unrounded P), the output's own (2^-8 |O|), and
# the fp32 scores: a sum of d <= 512 products errs by at most
# d 2^-24 sum|q k| scale, about 1e-3 at the tests' inputs (sum|q_i k_i| scale
# <= 35), which moves each P by that fraction: below another 2^-8 in all.
P_TOL = 2.0 ** -7
O_TOL = 2.0 ** -8
# LSE: the same score error, 512 * 2^-24 * 35 = 1.1e-3, plus fp32 roundings
LSE_TOL = 1.5e-3


# ----------------------------------------------------- plain definitions


def plain_tables(cached, new, free, table, page, T):
    table = [list(r) for r in table]
    slots, cu, taken = [], [0], 0
    for b, (c, n) in enumerate(zip(cached, new)):
        for pos in range(c, c + n):
            blk, off = divmod(pos, page)
            if off == 0:
                table[b][blk] = free[taken]
                taken += 1
            slots.append(table[b][blk] * page + off)
        cu.append(len(slots))
    return table, slots + [-1] * (T - len(slots)), cu, [c + n for c, n in zip(cached, new)], taken


def plain_attn(q, k, v, prefix_table, prefix_len, table, seq, cu, scale):
    """fp64 (O, LSE, sum_j P_j |v_j|) of the rows of requests, on the CPU; rows
    of no request are NaN."""
    T, H, d = q.shape
    page = k.shape[1]
    o = torch.full((T, H, d), math.nan, dtype=torch.float64)
    mag, lse = o.clone(), torch.full((T, H), math.nan, dtype=torch.float64)
    rows = lambda x, pages, n: x[pages[: -(-n // page)].long()].reshape(-1, d)[:n].double()
    kp, vp = (rows(x, prefix_table, prefix_len) for x in (k, v))
    for b, n in enumerate(seq):
        new = cu[b + 1] - cu[b]
        if new == 0:
            continue
        kk = torch.cat([kp, rows(k, table[b], n)])
        vv = torch.cat([vp, rows(v, table[b], n)])
        s = torch.einsum("ihd,jd->ihj", q[cu[b]:cu[b + 1]].double(), kk) * scale
        own = torch.arange(kk.shape[0]) - prefix_len
        last = (n - new + torch.arange(new)).clamp(min=-1)  # -1: the prefix alone
        seen = own[None, :] <= last[:, None]
        s = s.masked_fill(~seen[:, None, :], -math.inf)
        p = torch.softmax(s, -1).nan_to_num(0.0) if kk.shape[0] else s
        o[cu[b]:cu[b + 1]] = p @ vv
        mag[cu[b]:cu[b + 1]] = p @ vv.abs()
        lse[cu[b]:cu[b + 1]] = torch.logsumexp(s, -1)
    return o, lse, mag


class Case:
    """Inputs of one attention call on the CPU: new[b] query rows and seq[b]
    own tokens per request; every cache row that no one owns is NaN."""

    def __init__(self, new, seq, prefix, H, d, page, kv=2, pad=0, seed=1, extra=0,
                 qscale=2.0):
        g = torch.Generator().manual_seed(seed)
        self.new, self.seq, self.prefix = new, seq, prefix
        B, T = len(new), max(1, sum(new) + pad)
        n_own = [-(-n // page) for n in seq]
        n_pre = -(-prefix // page)
        n_pages = n_pre + sum(n_own) + 2
        width = max([1] + n_own) + extra
        perm = torch.randperm(n_pages, generator=g).to(torch.int32)
        self.prefix_table = perm[:n_pre].clone()
        self.table = torch.full((B, width), -1, dtype=torch.int32)
        at = n_pre
        live = torch.zeros(n_pages, page, dtype=torch.bool)

        def mark(pages, n):
            for i, p in enumerate(pages.tolist()):
                live[p, : min(page, n - i * page)] = True

        mark(self.prefix_table, prefix)
        for b in range(B):
            self.table[b, : n_own[b]] = perm[at: at + n_own[b]]
            mark(self.table[b, : n_own[b]], seq[b])
            at += n_own[b]

        def cache():
            x = torch.randn((n_pages, page, d), generator=g).to(BF)
            x[~live] = math.nan
            return x

        self.k = cache()
        self.v = self.k if kv == 1 else cache()
        self.kv = kv
        self.q = (qscale * torch.randn((T, H, d), generator=g)).to(BF)
        self.cu = np.concatenate([[0], np.cumsum(new)]).tolist()
        self.cfg = dsa.ServeConfig(n_pages=n_pages, max_tokens=T, batch=B, max_blocks=width,
                                   page_size=page, attn_heads=H, d_qk=d, d_v=d)

    def run(self, ws=None, o=None, lse=None, k=None):
        dv = lambda t: t.to(DEV)
        kd = dv(self.k) if k is None else k
        ws = dsa.serve_workspace(self.cfg, dsa.SERVE_WS_PREFIX, DEV) if ws is None else ws
        o, lse = dsa.prefix_attn(
            self.cfg, dv(self.q), kd, dv(self.prefix_table), self.prefix, dv(self.table),
            torch.tensor(self.seq, dtype=torch.int32, device=DEV),
            torch.tensor(self.cu, dtype=torch.int32, device=DEV),
            v_pages=None if self.kv == 1 else dv(self.v), o=o, lse=lse, ws=ws)
        torch.cuda.synchronize()
        return o.cpu(), lse.cpu(), dsa.get_device_status(ws)

    def plain(self):
        return plain_attn(self.q, self.k, self.v, self.prefix_table, self.prefix,
                          self.table, self.seq, self.cu, self.cfg.scale)


def check(got, ref, rows=None):
    o, lse = got[0].double(), got[1].double()
    ro, rl, mag = ref
    live = ~torch.isnan(rl[:, 0]) if rows is None else rows
    o, lse, ro, rl, mag = (x[live] for x in (o, lse, ro, rl, mag))
    assert torch.isfinite(o).all()
    empty = torch.isinf(rl)
    assert torch.equal(lse[empty], rl[empty]) and (o[empty] == 0).all()
    err = (o - ro).abs() - O_TOL * ro.abs() - P_TOL * mag
    assert (err <= 1e-30).all(), f"O: {err.max():.3g} over the bound"
    if (~empty).any():
        e = (lse - rl)[~empty].abs().max()
        assert e <= LSE_TOL + 2.0 ** -22 * rl[~empty].abs().max(), f"LSE: {e:.3g}"


# ------------------------------------------------------------ host checks


@pytest.fixture(scope="module")
def lib():
    dsa_build.build()
    return dsa._load()


def scfg(**kw):
    base = dict(n_pages=100, max_tokens=8, batch=4, max_blocks=10, page_size=64)
    base.update(kw)
    return dsa.ServeConfig(**base)


def test_serve_config_layout():
    C = dsa._CServeConfig
    assert ctypes.sizeof(C) == 48 and C.max_tokens.offset == 8
    assert C.page_size.offset == 16 and C.d_v.offset == 36 and C.sm_scale.offset == 40


def test_serve_config_is_copied_and_pickled_after_use():
    c = scfg()
    c._ref
    for d in (pickle.loads(pickle.dumps(c)), copy.copy(c), copy.deepcopy(c)):
        assert d == c and "_ref" not in vars(d)
        d._ref
    assert dataclasses.replace(c, batch=9)._ref._obj.batch == 9


@pytest.mark.parametrize("over,code", [
    (dict(n_pages=0), 1), (dict(max_tokens=0), 1), (dict(batch=0), 1),
    (dict(max_blocks=0), 1), (dict(page_size=0), 1), (dict(sm_scale=-1.0), 1),
    (dict(sm_scale=math.inf), 1), (dict(page_size=48), 2), (dict(page_size=256), 2),
    (dict(n_pages=1 << 25), 2), (dict(batch=65537), 2), (dict(max_blocks=1 << 24), 2),
    (dict(max_tokens=1 << 30), 2), (dict(d_qk=576), 2), (dict(d_v=256), 2),
    (dict(attn_heads=129), 2), (dict(attn_heads=0), 1), (dict(max_tokens=1 << 15), 2),
])
def test_invalid_serve_configs_rejected(lib, over, code):
    with pytest.raises(dsa.DsaError) as e:
        dsa.serve_workspace_size(scfg(**over), dsa.SERVE_WS_PREFIX)
    assert e.value.code == code


def test_serve_workspace_kinds(lib):
    # the tables and the append need the header alone, whatever the heads
    big = scfg(max_tokens=1 << 20, attn_heads=1000)
    assert dsa.serve_workspace_size(big, dsa.SERVE_WS_TABLES) == 256
    assert dsa.serve_workspace_size(big, dsa.SERVE_WS_APPEND) == 256
    assert dsa.serve_workspace_size(scfg(), dsa.SERVE_WS_PREFIX) >= 256
    for which in (-1, 3):
        with pytest.raises(dsa.DsaError) as e:
            dsa.serve_workspace_size(scfg(), which)
        assert e.value.code == 1


def test_serving_calls_check_arguments_before_launch(lib):
    cc = scfg().c()
    r = ctypes.byref(cc)
    p, off, ws = (ctypes.c_void_p(x) for x in (256, 264, 4096))
    nb = dsa.serve_workspace_size(scfg(), dsa.SERVE_WS_PREFIX)
    f = lib.dsa_build_page_tables
    assert f(r, p, p, p, 4, p, p, p, p, None, ws, 256, None) == 1
    assert f(r, p, p, None, 4, p, p, p, p, p, ws, 256, None) == 1     # no free list
    assert f(r, p, p, p, -1, p, p, p, p, p, ws, 256, None) == 1
    assert f(r, p, p, p, 4, p, off, p, p, p, ws, 256, None) == 4
    assert f(r, p, p, ctypes.c_void_p(258), 4, p, p, p, p, p, ws, 256, None) == 4
    assert f(r, p, p, p, 4, p, p, p, p, p, ws, 255, None) == 3
    assert f(r, p, p, p, 4, p, p, p, p, p, off, 256, None) == 4
    f = lib.dsa_append_cache
    k2 = ctypes.c_void_p(512)
    assert f(r, p, p, p, k2, None, ws, 256, None) == 1                # v_new alone
    assert f(r, p, p, None, k2, p, ws, 256, None) == 1                # v_pages alone
    assert f(r, p, p, p, k2, k2, ws, 256, None) == 1                  # one cache twice
    assert f(r, None, p, None, k2, None, ws, 256, None) == 1
    assert f(r, p, off, None, k2, None, ws, 256, None) == 4
    f = lib.dsa_prefix_attn
    assert f(r, p, p, p, None, 5, p, p, p, p, p, ws, nb, None) == 1   # prefix, no table
    assert f(r, p, p, p, p, -1, p, p, p, p, p, ws, nb, None) == 1
    assert f(r, p, p, p, p, 1 << 30, p, p, p, p, p, ws, nb, None) == 2
    assert f(r, p, p, p, p, 5, p, p, p, p, None, ws, nb, None) == 1
    assert f(r, p, p, p, p, 5, p, p, p, off, p, ws, nb, None) == 4
    assert f(r, p, p, p, p, 5, p, p, p, p, p, ws, nb - 1, None) == 3
    assert f(r, p, p, p, p, 5, p, p, p, p, p, None, nb, None) == 1


def test_serving_calls_refuse_what_overlaps(lib):
    """What a call writes may not meet what it reads, or itself; neighbours
    may touch."""
    c = scfg(max_tokens=512, d_qk=128, d_v=128)
    r, ws = ctypes.byref(c.c()), ctypes.c_void_p(1 << 24)
    at = {n: 4096 * (i + 1) for i, n in enumerate(
        ("cached", "new", "free", "table", "slots", "cu", "seq", "taken"))}
    size = dict(cached=16, new=16, free=400, table=160, slots=2048, cu=20, seq=16, taken=4)

    def tables(**over):
        a = [ctypes.c_void_p(x) for x in {**at, **over}.values()]
        return lib.dsa_build_page_tables(r, *a[:3], 100, *a[3:], ws, 256, None)

    for w in ("table", "slots", "cu", "seq", "taken"):
        for x in at:
            if x != w:
                assert tables(**{w: at[x]}) == 1, (w, x)             # the same place
                assert tables(**{w: at[x] + (size[x] - 1) // 16 * 16}) == 1, (w, x)  # its end
    page, row = 64, 256
    cache = c.n_pages * page * row
    at = dict(slots=1 << 20, k_new=2 << 20, v_new=3 << 20, k=1 << 30, v=2 << 30)

    def append(**over):
        a = [ctypes.c_void_p(x) for x in {**at, **over}.values()]
        return lib.dsa_append_cache(r, *a, ws, 256, None)

    for w in ("k", "v"):
        assert append(**{w: at["slots"] + 2032}) == 1
        assert append(**{w: at["k_new"] - cache + 16}) == 1
        assert append(**{w: at["v_new"] + 512 * row - 16}) == 1
    assert append(v=at["k"] + cache - 16) == 1
    assert append(k=at["v"] + cache - 16) == 1


def test_python_refuses_wrong_tensors():
    c = scfg()
    i = torch.zeros(4, dtype=torch.int32)
    with pytest.raises(ValueError):       # not on a GPU
        dsa.build_page_tables(c, i, i, i, torch.zeros(4, 10, dtype=torch.int32))
    with pytest.raises(TypeError):
        dsa.prefix_attn(c, None, None, None, 0, None, None, None)


# ------------------------------------------------------------ page tables


def tables_case(B, page, lo, hi, cached_hi, pad, seed):
    r = np.random.default_rng(seed)
    cached = r.integers(0, cached_hi + 1, B).tolist()
    new = r.integers(lo, hi + 1, B).tolist()
    have = [-(-c // page) for c in cached]
    need = [-(-(c + n) // page) for c, n in zip(cached, new)]
    n_pages = sum(need) + 5
    perm = r.permutation(n_pages).tolist()
    width = max([1] + need) + 1
    table, at = [], 0
    for b in range(B):
        table.append(perm[at:at + have[b]] + [-7] * (width - have[b]))
        at += have[b]
    cfg = dsa.ServeConfig(n_pages=n_pages, max_tokens=max(1, sum(new) + pad), batch=B,
                          max_blocks=width, page_size=page)
    return cfg, cached, new, perm[at:], table


def run_tables(cfg, cached, new, free, table, ws=None):
    i = lambda x: torch.tensor(x, dtype=torch.int32, device=DEV)
    ws = dsa.serve_workspace(cfg, dsa.SERVE_WS_TABLES, DEV) if ws is None else ws
    r = dsa.build_page_tables(cfg, i(cached), i(new), i(free), i(table), ws=ws)
    torch.cuda.synchronize()
    return [x.cpu().tolist() for x in r], dsa.get_device_status(ws)


@gpu
@pytest.mark.parametrize("B,page,lo,hi,cached_hi,pad", [
    (1, 64, 1, 1, 0, 0), (1, 16, 0, 0, 40, 2), (64, 64, 1, 1, 2048, 0),
    (255, 16, 0, 3, 100, 9), (256, 32, 1, 1, 31, 0), (257, 128, 0, 300, 500, 1),
    (1000, 16, 0, 40, 0, 0), (3, 16, 3000, 5000, 17, 100), (65536, 64, 0, 1, 63, 0)])
def test_page_tables(B, page, lo, hi, cached_hi, pad):
    cfg, cached, new, free, table = tables_case(B, page, lo, hi, cached_hi, pad, B + page)
    got, st = run_tables(cfg, cached, new, free, table)
    assert st == 0
    t, slots, cu, seq, taken = plain_tables(cached, new, free, table, page, cfg.max_tokens)
    assert got[0] == t and got[1] == slots and got[2] == cu and got[3] == seq
    assert got[4] == [taken]


@gpu
def test_page_tables_latch_what_is_wrong():
    i = dict(n_pages=20, batch=3, max_blocks=4, page_size=16)
    none = [[-1] * 4] * 3
    # a negative length, one past the table: no tokens for these requests
    cfg = dsa.ServeConfig(max_tokens=8, **i)
    got, st = run_tables(cfg, [-1, 60, 0], [2, 5, 3], [4, 5, 6], none)
    assert st == 7 and got[2] == [0, 0, 0, 3] and got[3] == [0, 0, 3]
    assert got[1] == [64, 65, 66] + [-1] * 5 and got[4] == [1]
    # the free list ends: later requests get -1, the need is reported
    got, st = run_tables(cfg, [0, 0, 0], [2, 3, 3], [4, 5], none)
    assert st == 10 and got[4] == [3]
    assert got[1] == [64, 65, 80, 81, 82, -1, -1, -1] and got[0][2][0] == -1
    # a page id outside the cache, in the free list and in a held entry
    got, st = run_tables(cfg, [0, 0, 0], [1, 1, 1], [4, 20, 5], none)
    assert st == 7 and got[1][:3] == [64, -1, 80]
    got, st = run_tables(cfg, [3, 0, 0], [1, 1, 0], [4], none)
    assert st == 7 and got[1][:2] == [-1, 64]
    # more tokens than slots
    cfg = dsa.ServeConfig(max_tokens=4, **i)
    got, st = run_tables(cfg, [0, 0, 0], [2, 3, 3], [4, 5, 6], none)
    assert st == 7 and got[2] == [0, 2, 4, 4] and got[1] == [64, 65, 80, 81]


# ----------------------------------------------------------------- append


@gpu
@pytest.mark.parametrize("T,d,page,kv", [(1, 128, 16, 2), (5, 512, 64, 1), (1023, 256, 128, 2),
                                         (4097, 512, 32, 2)])
def test_append(T, d, page, kv):
    g = torch.Generator().manual_seed(T)
    n_pages = T // page + 3
    cfg = dsa.ServeConfig(n_pages=n_pages, max_tokens=T, batch=1, max_blocks=1, page_size=page,
                          d_qk=d, d_v=d)
    slots = torch.randperm(n_pages * page, generator=g)[:T].to(torch.int32)
    slots[::7] = -1
    new = [torch.randn((T, d), generator=g).to(BF) for _ in range(kv)]
    pages = [torch.randn((n_pages, page, d), generator=g).to(BF) for _ in range(kv)]
    dev = [p.to(DEV) for p in pages]
    ws = dsa.serve_workspace(cfg, dsa.SERVE_WS_APPEND, DEV)
    dsa.append_cache(cfg, slots.to(DEV), new[0].to(DEV), dev[0],
                     v_new=new[1].to(DEV) if kv == 2 else None,
                     v_pages=dev[1] if kv == 2 else None, ws=ws)
    torch.cuda.synchronize()
    assert dsa.get_device_status(ws) == 0
    live = slots >= 0
    for n, p, got in zip(new, pages, dev):
        p.view(-1, d)[slots[live].long()] = n[live]
        assert torch.equal(got.cpu(), p)


@gpu
def test_append_skips_and_latches_a_slot_past_the_cache():
    cfg = dsa.ServeConfig(n_pages=2, max_tokens=3, batch=1, max_blocks=1, page_size=16, d_qk=128,
                          d_v=128)
    k = torch.zeros(2, 16, 128, dtype=BF, device=DEV)
    ws = dsa.serve_workspace(cfg, dsa.SERVE_WS_APPEND, DEV)
    dsa.append_cache(cfg, torch.tensor([31, 32, 0], dtype=torch.int32, device=DEV),
                     torch.ones(3, 128, dtype=BF, device=DEV), k, ws=ws)
    torch.cuda.synchronize()
    assert dsa.get_device_status(ws) == 7
    assert k.float().sum().item() == 2 * 128 and k[0, 0].min() == 1 and k[1, 15].min() == 1


# -------------------------------------------------------------- attention


@gpu
@pytest.mark.parametrize("d", [128, 256, 512])
@pytest.mark.parametrize("kv", [1, 2])
@pytest.mark.parametrize("page", [16, 32, 64, 128])
def test_attn_dims_and_pages(d, kv, page):
    check_case(Case([1, 1, 1], [1, 130, 77], 333, 16, d, page, kv, seed=d + page))


def check_case(c, **kw):
    got = c.run(**kw)
    assert got[2] == 0
    check(got, c.plain())
    return got


@gpu
@pytest.mark.parametrize("prefix", [0, 1, 15, 16, 17, 127, 128, 129, 255, 256, 257, 511, 513,
                                    5003])
def test_attn_prefix_lengths(prefix):
    check_case(Case([1, 1], [1, 256], prefix, 8, 512, 64, 1, seed=prefix))


@gpu
@pytest.mark.parametrize("H", [1, 3, 8, 64, 65, 127, 128])
def test_attn_heads(H):
    check_case(Case([1, 2, 1], [300, 2, 65], 700, H, 256, 32, 2, seed=H))


@gpu
@pytest.mark.parametrize("new,seq", [
    ([5, 0, 9, 1], [5, 40, 300, 1]),          # ragged, one request idle
    ([0, 0], [0, 17]),                        # no query row at all
    ([300], [300]),                           # a prompt's end, causal
    ([129, 70, 1], [700, 70, 513]),
    ([1] * 33, list(range(1, 34))),
    ([4, 3], [2, 0]),                         # rows before their own tokens
])
@pytest.mark.parametrize("prefix", [0, 300])
def test_attn_ragged_rows(new, seq, prefix):
    check_case(Case(new, seq, prefix, 8, 256, 16, 2, pad=3, seed=len(new)))


@gpu
def test_attn_many_rows_split_and_joined():
    """More row blocks than one wave, and few rows behind a long prefix."""
    check_case(Case([1] * 70, [3] * 70, 1500, 128, 128, 64, 2, seed=3))
    check_case(Case([1], [1], 40000, 1, 128, 128, 1, seed=4))


@gpu
def test_attn_peaked_and_shifted_scores():
    """Scores far from zero that grow along the keys (the running maximum is
    raised again and again) and rows where one key takes all."""
    c = Case([1, 1], [200, 31], 3000, 16, 512, 64, 2, seed=9, qscale=0.25)
    ramp = torch.linspace(-4, 4, 3000)
    page = c.cfg.page_size
    for j in range(3000):
        c.k[c.prefix_table[j // page].item(), j % page, :64] = ramp[j]
    c.q[:, :, :64] = 1.5
    check_case(c)
    c.q[:, 8:, :64] = -3.0
    check_case(c)


@gpu
def test_attn_leaves_other_rows_and_repeats():
    c = Case([2, 0, 3], [70, 5, 3], 600, 16, 512, 64, 1, pad=4, seed=11)
    o = torch.full((9, 16, 512), 7.0, dtype=BF, device=DEV)
    lse = torch.full((9, 16), 7.0, device=DEV)
    a = check_case(c, o=o, lse=lse)
    assert (a[0][5:] == 7).all() and (a[1][5:] == 7).all()
    for _ in range(3):
        b = c.run()
        assert torch.equal(a[0][:5], b[0][:5]) and torch.equal(a[1][:5], b[1][:5])


@gpu
def test_attn_infinities_and_nan_in_unseen_places():
    """Unowned rows hold NaN in every case; here also infinities, and a table
    whose unread entries are out of range."""
    c = Case([1, 3], [65, 30], 130, 16, 512, 64, 2, seed=5, extra=2)
    c.k[torch.isnan(c.k)] = math.inf
    c.v[torch.isnan(c.v)] = -math.inf
    c.table[c.table < 0] = 1 << 30
    check_case(c)


@gpu
def test_attn_latches_bad_pages_and_lengths():
    for spoil in ("prefix", "table", "seq", "cu", "cu0"):
        c = Case([1, 1], [20, 90], 100, 16, 512, 64, 1, seed=6)
        if spoil == "prefix":
            c.prefix_table[1] = c.cfg.n_pages
        elif spoil == "table":
            c.table[1, 1] = -1
        elif spoil == "seq":
            c.seq = [20, 64 * c.cfg.max_blocks + 1]
        elif spoil == "cu":
            c.cu = [0, 1, 3]
        else:
            c.cu = [-1, 1, 2]
        assert c.run()[2] == 7, spoil
        # the workspace serves the next call as before
        check_case(Case([1, 1], [20, 90], 100, 16, 512, 64, 1, seed=6))


@gpu
def test_attn_on_a_side_stream_and_in_a_graph():
    c = Case([1, 2], [40, 300], 500, 16, 512, 64, 1, seed=8)
    ref = c.plain()
    dv = lambda t: t.to(DEV)
    q, k, pt, tb = dv(c.q), dv(c.k), dv(c.prefix_table), dv(c.table)
    seq = torch.tensor(c.seq, dtype=torch.int32, device=DEV)
    cu = torch.tensor(c.cu, dtype=torch.int32, device=DEV)
    ws = dsa.serve_workspace(c.cfg, dsa.SERVE_WS_PREFIX, DEV)
    o = torch.zeros((3, 16, 512), dtype=BF, device=DEV)
    lse = torch.zeros((3, 16), device=DEV)
    torch.cuda.synchronize()
    call = lambda: dsa.prefix_attn(c.cfg, q, k, pt, c.prefix, tb, seq, cu, o=o, lse=lse, ws=ws)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        call()
    torch.cuda.synchronize()
    check((o.cpu(), lse.cpu()), ref)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    # new lengths and values in the captured buffers
    c2 = Case([2, 1], [40, 300], 500, 16, 512, 64, 1, seed=8)
    q.copy_(c2.q * 0.5)
    c2.q = (c2.q * 0.5).to(BF)
    cu.copy_(torch.tensor(c2.cu, dtype=torch.int32))
    o.zero_()
    for _ in range(2):
        g.replay()
    torch.cuda.synchronize()
    assert dsa.get_device_status(ws) == 0
    check((o.cpu(), lse.cpu()), c2.plain())


@gpu
@pytest.mark.parametrize("at", [300, 5, 255, 256, 700, 1999])
@pytest.mark.parametrize("jump", [15.0, 30.0, 120.0, 5000.0])
def test_attn_scores_far_beyond_the_first_reference(at, jump):
    """One key (and a few after it) whose score passes everything before by up
    to thousands: exact scores, so the bound stays that of P's rounding.  Some
    rows have the jump, some its negative, some none."""
    c = Case([1, 1], [40, 300], 2000, 16, 512, 64, 2, seed=at)
    c.cfg = dataclasses.replace(c.cfg, sm_scale=1.0)
    c.q[:] = 0
    c.q[:, :, 0] = 1.0
    c.q[:, 5::3, 0] = -1.0
    c.q[:, 6::3, 0] = 0.0
    live = ~torch.isnan(c.k)
    c.k = torch.where(live, (2 * torch.rand(c.k.shape, generator=torch.Generator().manual_seed(1))
                             ).round().to(BF), c.k)
    page = c.cfg.page_size
    for n, j in enumerate(range(at, min(at + 3, 2000))):
        c.k[c.prefix_table[j // page].item(), j % page, 0] = jump * (1 + n)
    # the last own token of request 1 passes that again
    c.k[c.table[1, 299 // page].item(), 299 % page, 0] = 4 * jump
    check_case(c)


@gpu
def test_attn_large_values_and_scales():
    c = Case([1, 2], [30, 300], 600, 16, 256, 32, 2, seed=21)
    c.cfg = dataclasses.replace(c.cfg, sm_scale=0.01)
    c.v = (c.v.float() * 1e30).to(BF)
    check_case(c)


@gpu
def test_attn_shares_that_begin_inside_units():
    """384 and 1152 rows behind a prefix of odd length: shares that begin and
    end inside units, whose tiles are taken from the middle on."""
    check_case(Case([3], [40], 30011, 128, 128, 64, 1, seed=31))
    check_case(Case([2, 1, 6], [2, 300, 77], 9999, 128, 128, 16, 2, seed=32))


@gpu
@pytest.mark.parametrize("B,H", [(1000, 8), (3000, 1)])
def test_attn_many_requests(B, H):
    """More requests than threads in a block; some idle, some without own
    tokens before this step."""
    r = np.random.default_rng(B)
    new = r.integers(0, 3, B).tolist()
    seq = [n + int(x) for n, x in zip(new, r.integers(0, 20, B))]
    check_case(Case(new, seq, 70, H, 128, 16, 2, pad=5, seed=B))


@gpu
@pytest.mark.parametrize("live", [[0], [2046], [31, 32, 33, 64, 1000, 1031, 2047],
                                  [1, 30, 63, 65, 95, 97, 500, 501, 2000]])
def test_attn_idle_requests_between(live):
    """A batch that is mostly idle, some of it with tokens but no query."""
    new, seq = [0] * 2048, [0, 5] * 1024
    for b in live:
        new[b], seq[b] = 1 + b % 3, 40 + b % 300
    check_case(Case(new, seq, 0, 8, 128, 16, 2, seed=len(live)))
    check_case(Case(new, seq, 300, 8, 128, 16, 2, seed=len(live)))


@gpu
@pytest.mark.parametrize("B,new,H,prefix", [(3, 2720, 128, 300), (65536, 1, 16, 40),
                                            (65536, 0, 16, 40)])
def test_attn_largest_row_counts(B, new, H, prefix):
    """Up to 2^20 rows and 65536 requests (one in seven idle, or all but two);
    64 rows are compared."""
    d, page = 128, 16
    r = np.random.default_rng(B + new)
    news = np.where(np.arange(B) % 7 == 3, 0, new) if B > 3 else np.full(B, new)
    if new == 0:
        news[[5, B - 1]] = [3, 1000]
    seqs = news + r.integers(0, 20, B)
    cu = np.concatenate([[0], np.cumsum(news)])
    own = -(-seqs // page)
    width, n_pre = int(own.max()), -(-prefix // page)
    n_pages = n_pre + int(own.sum())
    table = np.full((B, width), -1, dtype=np.int32)
    table[np.arange(width)[None] < own[:, None]] = n_pre + np.arange(int(own.sum()))
    T = (1 << 20) // H
    g = torch.Generator(device=DEV).manual_seed(B + new)
    rand = lambda *n: torch.randn(n, generator=g, device=DEV, dtype=BF)
    q, k, v = 2 * rand(T, H, d), rand(n_pages, page, d), rand(n_pages, page, d)
    cfg = dsa.ServeConfig(n_pages=n_pages, max_tokens=T, batch=B, max_blocks=width,
                          page_size=page, attn_heads=H, d_qk=d, d_v=d)
    i32 = lambda x: torch.tensor(np.asarray(x), dtype=torch.int32, device=DEV)
    ws = dsa.serve_workspace(cfg, dsa.SERVE_WS_PREFIX)
    o, lse = dsa.prefix_attn(cfg, q, k, i32(np.arange(n_pre)), prefix, i32(table), i32(seqs),
                             i32(cu), v_pages=v, ws=ws)
    assert dsa.get_device_status(ws) == 0
    n = int(cu[-1])
    for t in sorted({0, n - 1, *r.integers(0, n, 62).tolist()}):
        b = int(np.searchsorted(cu, t, side="right")) - 1
        keys = int(seqs[b] - news[b] + t - cu[b] + 1)
        rows = lambda x: torch.cat([
            x[:n_pre].reshape(-1, d)[:prefix],
            x[i32(table[b, : own[b]]).long()].reshape(-1, d)[:keys]]).double().cpu()
        kk, vv = rows(k), rows(v)
        sc = q[t].double().cpu() @ kk.T * cfg.scale
        p = torch.softmax(sc, -1)
        ref, mag = p @ vv, p @ vv.abs()
        err = (o[t].double().cpu() - ref).abs()
        assert (err <= P_TOL * mag + O_TOL * ref.abs()).all(), (t, b)
        assert (lse[t].double().cpu() - torch.logsumexp(sc, -1)).abs().max() <= LSE_TOL
    assert not o[n:].any() and not lse[n:].any()


@gpu
@pytest.mark.parametrize("captured", [False, True])
def test_append_sees_what_the_stream_wrote_before(captured):
    """Slots and rows that a kernel or a copy writes right before the call,
    which is launched early, and that are overwritten right behind it."""
    T, d, n_pages = 1023, 256, 80
    cfg = dsa.ServeConfig(n_pages=n_pages, max_tokens=T, batch=1, max_blocks=1, page_size=16,
                          d_qk=d, d_v=d)
    g = torch.Generator(device=DEV).manual_seed(1)
    ws = dsa.serve_workspace(cfg, dsa.SERVE_WS_APPEND)
    slots = torch.full((T,), -1, dtype=torch.int32, device=DEV)
    rows = torch.zeros((T, d), dtype=BF, device=DEV)
    pages = [torch.zeros((n_pages, 16, d), dtype=BF, device=DEV) for _ in range(4)]
    where = [torch.randperm(n_pages * 16, generator=g, device=DEV)[:T].to(torch.int32)
             for _ in pages]
    what = [torch.randn((T, d), generator=g, device=DEV).to(BF) for _ in pages]

    def steps():
        for i, p in enumerate(pages):
            rows.copy_(what[i])
            torch.add(where[i], 0, out=slots)
            dsa.append_cache(cfg, slots, rows, p, ws=ws)
            slots.fill_(-1)
            rows.zero_()

    steps()
    torch.cuda.synchronize()
    for p in pages:
        p.zero_()
    if captured:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            steps()
        for _ in range(10):
            graph.replay()
    else:
        for _ in range(10):
            steps()
    for p, s, x in zip(pages, where, what):
        ref = torch.zeros_like(p).view(-1, d)
        ref[s.long()] = x
        assert torch.equal(p.view(-1, d), ref)
    assert dsa.get_device_status(ws) == 0


@gpu
@pytest.mark.parametrize("captured", [False, True])
def test_attn_sees_what_the_stream_wrote_before(captured):
    """Lengths, tables and rows that a copy, a fill, a kernel or another stream
    writes right before the call, which is launched early, and outputs that
    are read and inputs that are overwritten right behind it."""
    cases = [Case([1, 2], [40, 300], 500, 16, 512, 64, 1, seed=8),
             Case([2, 1], [7, 900], 500, 16, 512, 64, 1, seed=9)]
    size = max(c.table.numel() for c in cases), max(c.cfg.n_pages for c in cases)
    for c in cases:
        c.cfg = dataclasses.replace(c.cfg, max_blocks=15, n_pages=size[1])
        c.table = torch.nn.functional.pad(c.table, (0, 15 - c.table.shape[1]), value=-1)
        c.k = torch.cat([c.k, c.k[:1].expand(size[1] - c.k.shape[0], -1, -1)])
    cfg = cases[0].cfg
    refs = [c.plain() for c in cases]
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=DEV)
    src = [(i32(c.seq), i32(c.cu), c.table.to(DEV), c.prefix_table.to(DEV), c.q.to(DEV),
            c.k.to(DEV)) for c in cases]
    seq, cu, table, ptable, q, k = (torch.zeros_like(t) for t in src[0])
    outs = [(torch.zeros(3, 16, 512, dtype=BF, device=DEV), torch.zeros(3, 16, device=DEV))
            for _ in cases]
    o, lse = torch.zeros_like(outs[0][0]), torch.zeros_like(outs[0][1])
    ws = dsa.serve_workspace(cfg, dsa.SERVE_WS_PREFIX)
    side = torch.cuda.Stream()

    def call():
        dsa.prefix_attn(cfg, q, k, ptable, 500, table, seq, cu, o=o, lse=lse, ws=ws)

    def step(i, last):
        s, c, t, p, x, y = src[i]
        for dst, new in ((k, y), (q, x), (table, t), (ptable, p), (seq, s), (cu, c)):
            if dst is not last:
                dst.copy_(new)
        here = torch.cuda.current_stream()
        if last is seq:          # from another stream
            side.wait_stream(here)
            with torch.cuda.stream(side):
                seq.copy_(s)
            here.wait_stream(side)
        elif last is cu:         # by a kernel
            torch.add(c, 0, out=cu)
        else:
            last.copy_(dict(q=x, k=y)["q" if last is q else "k"])
        call()
        outs[i][0].copy_(o)
        outs[i][1].copy_(lse)
        seq.fill_(-7)            # behind it: nothing of the call may see this
        cu.zero_()

    for last in (seq, cu, q, k):
        for out in outs:
            out[0].zero_(), out[1].zero_()
        if captured:
            step(0, last)
            torch.cuda.synchronize()
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g):
                step(0, last)
                step(1, last)
            for _ in range(20):
                g.replay()
        else:
            for _ in range(20):
                step(0, last)
                step(1, last)
        assert dsa.get_device_status(ws) == 0
        for out, ref in zip(outs, refs):
            check((out[0].cpu(), out[1].cpu()), ref)


@gpu
def test_attn_padding_rows_may_hold_anything():
    c = Case([2, 1], [70, 5], 300, 16, 512, 64, 1, pad=9, seed=12)
    c.q[3:] = math.nan
    check_case(c)
    c.q[3:] = math.inf
    check_case(c)


@gpu
def test_cache_beyond_32_bit_offsets():
    """A cache of 5 GiB whose last pages are used: byte offsets past 2^32."""
    page, d, n_pages = 128, 512, 40960
    k = torch.zeros((n_pages, page, d), dtype=BF, device=DEV)
    c = Case([1, 1], [100, 130], 300, 16, d, page, 1, seed=41)
    far = n_pages - c.cfg.n_pages
    k[far:] = c.k.to(DEV)
    c.prefix_table += far
    c.table[c.table >= 0] += far
    c.cfg = dataclasses.replace(c.cfg, n_pages=n_pages)
    ref = plain_attn(c.q, c.k, c.v, c.prefix_table - far, c.prefix,
                     torch.where(c.table >= 0, c.table - far, c.table), c.seq, c.cu, c.cfg.scale)
    got = c.run(k=k)
    assert got[2] == 0
    check(got, ref)
    # and the append to the cache's last rows
    ac = dsa.ServeConfig(n_pages=n_pages, max_tokens=3, batch=1, max_blocks=1, page_size=page)
    slots = torch.tensor([n_pages * page - 1, -1, n_pages * page - 200], dtype=torch.int32,
                         device=DEV)
    new = torch.randn(3, d, device=DEV).to(BF)
    dsa.append_cache(ac, slots, new, k)
    assert torch.equal(k.view(-1, d)[-1], new[0]) and torch.equal(k.view(-1, d)[-200], new[2])


@gpu
def test_attn_two_calls_at_once():
    """Two streams, a workspace each."""
    cs = [Case([1, 2], [40, 300], 3000, 16, 512, 64, 1, seed=51),
          Case([1] * 9, [33] * 9, 2000, 64, 256, 32, 2, seed=52)]
    streams = [torch.cuda.Stream() for _ in cs]
    ins = []
    dv = lambda t: t.to(DEV)
    for c in cs:
        i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=DEV)
        k = dv(c.k)
        ins.append((dv(c.q), k, dv(c.prefix_table), dv(c.table), i32(c.seq), i32(c.cu),
                    None if c.kv == 1 else dv(c.v),
                    dsa.serve_workspace(c.cfg, dsa.SERVE_WS_PREFIX, DEV)))
    torch.cuda.synchronize()
    outs = [None, None]
    for _ in range(5):
        for x, (c, s) in enumerate(zip(cs, streams)):
            q, k, pt, tb, seq, cu, v, ws = ins[x]
            with torch.cuda.stream(s):
                outs[x] = dsa.prefix_attn(c.cfg, q, k, pt, c.prefix, tb, seq, cu, v_pages=v, ws=ws)
    torch.cuda.synchronize()
    for c, (o, lse), i in zip(cs, outs, ins):
        assert dsa.get_device_status(i[-1]) == 0
        check((o.cpu(), lse.cpu()), c.plain())


# ------------------------------------------------- the calls as one engine


@gpu
@pytest.mark.parametrize("kv,page,d", [(1, 64, 512), (2, 16, 128)])
def test_serving_steps_together(kv, page, d):
    """A prompt goes into the cache once; three requests then grow by ragged
    steps (tables -> append -> attention); each step's rows equal dense
    attention over prompt + own tokens in fp64."""
    g = torch.Generator().manual_seed(17)
    B, H, P, n_pages, width, T = 3, 8, 300, 64, 12, 40
    bf = lambda *s: torch.randn(s, generator=g).to(BF)
    cfg = dsa.ServeConfig(n_pages=n_pages, max_tokens=T, batch=B, max_blocks=width,
                          page_size=page, attn_heads=H, d_qk=d, d_v=d)
    caches = [torch.full((n_pages, page, d), math.nan, dtype=BF, device=DEV) for _ in range(kv)]
    perm = torch.randperm(n_pages, generator=g).to(torch.int32)
    n_pre = -(-P // page)
    ws = [dsa.serve_workspace(cfg, w, DEV) for w in range(3)]
    ptab = perm[:n_pre].to(DEV)
    prompt = [bf(P, d) for _ in range(kv)]
    slots = (ptab.cpu()[torch.arange(P) // page] * page + torch.arange(P) % page).to(torch.int32)
    pc = dsa.ServeConfig(n_pages=n_pages, max_tokens=P, batch=1, max_blocks=1, page_size=page,
                         d_qk=d, d_v=d)
    two = lambda xs: xs[1] if kv == 2 else None
    dsa.append_cache(pc, slots.to(DEV), prompt[0].to(DEV), caches[0],
                     v_new=prompt[1].to(DEV) if kv == 2 else None, v_pages=two(caches))
    free = perm[n_pre:].to(DEV)
    table = torch.full((B, width), -1, dtype=torch.int32, device=DEV)
    lens = torch.zeros(B, dtype=torch.int32, device=DEV)
    own = [[torch.zeros(0, d, dtype=BF) for _ in range(B)] for _ in range(kv)]
    for new in ([7, 20, 1], [1, 1, 1], [0, 15, 16], [1, 0, 1]):
        nl = torch.tensor(new, dtype=torch.int32, device=DEV)
        r = dsa.build_page_tables(cfg, lens, nl, free, table, ws=ws[0])
        rows = [bf(T, d) for _ in range(kv)]
        dsa.append_cache(cfg, r.slot_map, rows[0].to(DEV), caches[0],
                         v_new=rows[1].to(DEV) if kv == 2 else None, v_pages=two(caches),
                         ws=ws[1])
        q = bf(T, H, d)
        o, lse = dsa.prefix_attn(cfg, q.to(DEV), caches[0], ptab, P, table, r.seq_lens,
                                 r.cu_tokens, v_pages=two(caches), ws=ws[2])
        free = free[int(r.pages_taken):]    # a slice of the list
        lens = r.seq_lens.clone()
        torch.cuda.synchronize()
        assert [dsa.get_device_status(w) for w in ws] == [0, 0, 0]
        cu = np.concatenate([[0], np.cumsum(new)]).tolist()
        for b in range(B):
            for x in range(kv):
                own[x][b] = torch.cat([own[x][b], rows[x][cu[b]:cu[b + 1]]])
            n = own[0][b].shape[0]
            kk = torch.cat([prompt[0], own[0][b]]).double()
            vv = torch.cat([prompt[-1], own[-1][b]]).double()
            for i in range(new[b]):
                t, m = cu[b] + i, P + n - new[b] + i + 1
                s = q[t].double() @ kk[:m].T * cfg.scale
                p = torch.softmax(s, -1)
                check((o[t:t + 1].cpu(), lse[t:t + 1].cpu()),
                      ((p @ vv[:m])[None], torch.logsumexp(s, -1)[None],
                       (p @ vv[:m].abs())[None]))
        assert (o[cu[-1]:] == 0).all()


@gpu
def test_serving_step_in_a_graph():
    """Tables, append and attention of one step, captured once and replayed
    on new lengths, rows and free pages."""
    B, H, P, page, d, n_pages, width, T = 2, 16, 200, 32, 256, 40, 10, 12
    cfg = dsa.ServeConfig(n_pages=n_pages, max_tokens=T, batch=B, max_blocks=width,
                          page_size=page, attn_heads=H, d_qk=d, d_v=d)
    g = torch.Generator().manual_seed(3)
    bf = lambda *s: torch.randn(s, generator=g).to(BF).to(DEV)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=DEV)
    k = bf(n_pages, page, d)
    ptab = i32(list(range(7)))
    ws = [dsa.serve_workspace(cfg, w, DEV) for w in range(3)]
    table = torch.full((B, width), -1, dtype=torch.int32, device=DEV)
    lens, new, free = i32([0, 0]), i32([5, 3]), i32(list(range(39, 6, -1)))
    rows, q = bf(T, d), bf(T, H, d)
    out = dsa.PageTables(table, *(torch.zeros(n, dtype=torch.int32, device=DEV)
                                  for n in (T, B + 1, B, 1)))
    o = torch.zeros((T, H, d), dtype=BF, device=DEV)
    lse = torch.zeros((T, H), device=DEV)

    def step():
        dsa.build_page_tables(cfg, lens, new, free, table, out=out, ws=ws[0])
        dsa.append_cache(cfg, out.slot_map, rows, k, ws=ws[1])
        dsa.prefix_attn(cfg, q, k, ptab, P, table, out.seq_lens, out.cu_tokens, o=o, lse=lse,
                        ws=ws[2])

    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        step()
    torch.cuda.synchronize()
    table.fill_(-1)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    held, taken = [0, 0], 0
    for n in ([5, 3], [1, 1], [0, 12], [4, 0]):
        new.copy_(i32(n))
        lens.copy_(i32(held))
        free.copy_(i32((list(range(39, 6, -1))[taken:] + [0] * 33)[:33]))
        rows.copy_(bf(T, d))
        q.copy_(bf(T, H, d))
        graph.replay()
        torch.cuda.synchronize()
        assert [dsa.get_device_status(w) for w in ws] == [0, 0, 0]
        taken += int(out.pages_taken)
        held = [a + b for a, b in zip(held, n)]
        assert out.seq_lens.tolist() == held
        cu = out.cu_tokens.tolist()
        slots = out.slot_map.tolist()
        for x in range(cu[-1]):
            assert torch.equal(k.view(-1, d)[slots[x]], rows[x])
        ref = plain_attn(q.cpu(), k.cpu(), k.cpu(), ptab.cpu(), P, table.cpu(), held, cu, cfg.scale)
        check((o.cpu(), lse.cpu()), ref)


CHECKS_CHILD = r"""
import json, sys
import numpy as np, torch
sys.path.insert(0, {root!r})
import long_context_sparse_gb300 as dsa
from tests.test_serving import Case, tables_case, run_tables
out, status = {{}}, []
for x, c in enumerate((Case([1, 3, 0], [50, 300, 7], 700, 16, 512, 64, 1, pad=2, seed=1),
                       Case([2] * 5, [9] * 5, 300, 8, 128, 16, 2, seed=2),
                       Case([1], [33], 20000, 64, 256, 128, 2, seed=3))):
    o, lse, st = c.run()
    out["o%d" % x], out["lse%d" % x] = o.float().numpy(), lse.numpy()
    status.append(st)
got, st = run_tables(*tables_case(300, 16, 0, 40, 50, 3, 5))
status.append(st)
out["tables"] = np.array(got[1])
np.savez(sys.argv[1], **out)
print(json.dumps({{"library": dsa.library_path(), "status": status}}))
"""


@gpu
def test_serving_in_the_checks_build(tmp_path):
    """The bounds-checking build runs the serving calls clean and agrees bit
    for bit."""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    runs = []
    for checks in ("1", "0"):
        path = str(tmp_path / f"c{checks}.npz")
        r = subprocess.run([sys.executable, "-c", CHECKS_CHILD.format(root=root), path],
                           env=dict(os.environ, DSA_GB300_CHECKS=checks), cwd=root,
                           capture_output=True, text=True, timeout=600)
        assert r.returncode == 0, r.stderr[-2000:]
        info = json.loads(r.stdout.strip().splitlines()[-1])
        assert info["status"] == [0, 0, 0, 0]
        assert info["library"].endswith("_checks.so") == (checks == "1")
        runs.append(np.load(path))
    for key in runs[0].files:
        assert np.array_equal(runs[0][key], runs[1][key]), key
