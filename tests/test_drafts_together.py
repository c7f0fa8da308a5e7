"""Drafting, weighing and forgetting as a serving loop has them, behind kernels
that write late, side by side, and in the checks build."""
import json
import math
import os
import subprocess
import sys
import types

import pytest
import torch

import long_context_sparse_gb300 as dsa
from tests.test_evict import Evict, check_evict, plain_keep, same
from tests.test_logprobs import logits_of
from tests.test_serving import BF, DEV, Case, check
from tests.test_serving_early import late, replayed  # noqa: F401 (a fixture)
from tests.test_tree import (check_tree, i32, plain_bits, plain_tree, plain_weights, signed,
                             tree_parents, weights_case)

gpu = pytest.mark.gpu


# ------------------------------------------------------- a serving loop


@gpu
@pytest.mark.parametrize("kv", [1, 2])
def test_draft_accept_weigh_and_forget(kv):
    """Several steps of a group: tables, append, tree, attention, weights, the
    rejected drafts dropped, the cache kept within a budget, its pages handed back.
    Each call is checked on what the calls before it left."""
    B, H, d, page, P, width, budget = 3, 16, 128, 16, 200, 12, 20
    g = torch.Generator().manual_seed(kv)
    n_pages = -(-P // page) + B * width + 2
    perm = torch.randperm(n_pages, generator=g).tolist()
    prefix_table = perm[: -(-P // page)]
    free = perm[len(prefix_table):]
    bf = lambda *s: torch.randn(s, generator=g).to(BF)
    cache = [bf(n_pages, page, d).to(DEV) for _ in range(kv)]
    w = torch.full((n_pages, page), math.nan, device=DEV)     # new tokens start from nothing
    table = torch.full((B, width), -1, dtype=torch.int32, device=DEV)
    lens = [0, 0, 0]
    peak = 0
    for step in range(9):
        new = [int(x) for x in torch.randint(0, 30, (B,), generator=g)]
        if step == 4:
            new[1] = 0
        T = max(1, sum(new) + 2)
        cfg = dsa.ServeConfig(n_pages=n_pages, max_tokens=T, batch=B, max_blocks=width,
                              page_size=page, attn_heads=H, d_qk=d, d_v=d)
        space = lambda which: dsa.serve_workspace(cfg, which, DEV)
        ws = {x: space(x) for x in (dsa.SERVE_WS_TABLES, dsa.SERVE_WS_APPEND, dsa.SERVE_WS_PREFIX,
                                    dsa.SERVE_WS_TREE, dsa.SERVE_WS_WEIGHTS, dsa.SERVE_WS_EVICT)}
        free_d = i32(free)
        t = dsa.build_page_tables(cfg, i32(lens), i32(new), free_d, table,
                                  ws=ws[dsa.SERVE_WS_TABLES])
        taken = t.pages_taken.item()
        free = free[taken:]
        rows = [bf(T, d).to(DEV) for _ in range(kv)]
        dsa.append_cache(cfg, t.slot_map, rows[0], cache[0], v_new=rows[1] if kv == 2 else None,
                         v_pages=cache[1] if kv == 2 else None, ws=ws[dsa.SERVE_WS_APPEND])
        parents = tree_parents(new, "random", step) + [-1] * (T - sum(new))
        bits = dsa.build_tree(cfg, i32(parents), t.cu_tokens, words=1, ws=ws[dsa.SERVE_WS_TREE])
        q = (2 * torch.randn((T, H, d), generator=g)).to(BF)
        ptab = i32(prefix_table)
        o, lse = dsa.tree_attn(cfg, q.to(DEV), cache[0], ptab, P, table, t.seq_lens, t.cu_tokens,
                               bits, v_pages=cache[1] if kv == 2 else None,
                               ws=ws[dsa.SERVE_WS_PREFIX])
        cu, seq = t.cu_tokens.tolist(), t.seq_lens.tolist()
        assert seq == [a + b for a, b in zip(lens, new)]
        plain = plain_bits(parents, cu, T, 1)
        assert torch.equal(bits.cpu()[: cu[-1]], signed(plain)[: cu[-1]])
        host = types.SimpleNamespace(q=q, k=cache[0].cpu(), v=cache[-1].cpu(), prefix=P, seq=seq,
                                     prefix_table=ptab.cpu(), cu=cu, table=table.cpu(), cfg=cfg)
        if cu[-1]:
            check([o.cpu(), lse.cpu()], plain_tree(host, plain))
        old = w.clone()
        dsa.key_weights(cfg, q.to(DEV), lse, cache[0], table, t.seq_lens, t.cu_tokens, w,
                        tree_bits=bits, decay=0.9, ws=ws[dsa.SERVE_WS_WEIGHTS])
        want, tol = plain_weights(host, plain, lse.cpu(), old.cpu(), old.cpu(), 0.9)
        live = ~torch.isnan(want)
        assert torch.equal(torch.isnan(w.cpu().view(-1)), ~live)
        assert ((w.cpu().double().view(-1) - want).abs() <= tol)[live].all()
        # a path of each tree is accepted
        slots = lambda b, n: torch.tensor(
            [int(table[b, p // page]) * page + p % page for p in range(n)], dtype=torch.long)
        rank = torch.full((n_pages, page), math.inf)
        keep = []
        for b in range(B):
            path, at = [], new[b] - 1 - int(new[b] > 3)
            while at >= 0:
                path.append(at)
                at = parents[cu[b] + at]
            s = slots(b, seq[b])
            for j in range(new[b]):
                if j not in path:
                    rank.view(-1)[s[lens[b] + j]] = -math.inf
            keep.append(lens[b] + len(path))
        for ranks, keeps, first, last in ((rank, keep, 0, 0), (None, [budget] * B, 2, 6)):
            before = [x.cpu() for x in cache] + [w.cpu()]
            dsa.evict_cache(cfg, w, table, i32(seq), i32(keeps), cache[0],
                            v_pages=cache[1] if kv == 2 else None, n_first=first, n_last=last,
                            ws=ws[dsa.SERVE_WS_EVICT],
                            rank_pages=None if ranks is None else ranks.to(DEV))
            r = dsa.release_pages(cfg, i32(seq), i32(keeps), table, ws=ws[dsa.SERVE_WS_TABLES])
            gone = []
            for b in range(B):
                s = slots(b, seq[b])
                left = min(seq[b], keeps[b])
                by = (before[-1] if ranks is None else ranks).view(-1)[s].tolist()
                src = plain_keep(by, left, first, last)
                for x, y in zip(before[:-1], cache):
                    assert torch.equal(y.view(-1, d)[s[:left].to(DEV)].cpu(),
                                       x.view(-1, d)[s[src]])
                assert same(w.view(-1)[s[:left].to(DEV)].cpu(), before[-1].view(-1)[s[src]])
                gone += table[b, -(-left // page): -(-seq[b] // page)].tolist()
            seq = r.new_lens.tolist()
            n = r.n_released.item()
            assert r.pages[:n].tolist() == gone
            free += gone
        lens = seq
        peak = max(peak, max(lens))
        for x in ws.values():
            assert dsa.get_device_status(x) == 0
        held = sum(-(-n // page) for n in lens)
        assert len(set(free)) == len(free) == n_pages - len(prefix_table) - held
    assert peak == budget


@gpu
def test_a_step_in_a_graph():
    """Tree, attention, weights, eviction, release and log-probs in one graph; each
    replay on the same inputs gives what the calls one by one give."""
    c = Case([6, 20], [100, 230], 300, 16, 128, 16, 2, seed=3)
    dv = lambda t: t.to(DEV)
    parents = i32(tree_parents(c.new, "random", 3))
    q, table, seq, cu, ptab = dv(c.q), dv(c.table), i32(c.seq), i32(c.cu), dv(c.prefix_table)
    k0, v0 = dv(torch.nan_to_num(c.k)), dv(torch.nan_to_num(c.v))
    w0 = torch.rand(c.k.shape[:2], device=DEV)
    head = (torch.randn(26, 16 * 128, device=DEV) * 0.02).to(BF)
    logits, tok = logits_of(26, 5000, BF, 4)
    k, v, w = k0.clone(), v0.clone(), w0.clone()
    keep = i32([60, 300])
    ws = {x: dsa.serve_workspace(c.cfg, x, DEV) for x in (dsa.SERVE_WS_PREFIX, dsa.SERVE_WS_TREE,
                                                          dsa.SERVE_WS_WEIGHTS,
                                                          dsa.SERVE_WS_EVICT,
                                                          dsa.SERVE_WS_TABLES)}
    lws = dsa.logprobs_workspace(DEV)
    bits = torch.zeros((26, 1), dtype=torch.int32, device=DEV)
    o, lse = torch.zeros_like(q), torch.zeros(q.shape[:2], device=DEV)
    rel = dsa.ReleasedPages(torch.zeros(2, dtype=torch.int32, device=DEV),
                            torch.full((50,), -1, dtype=torch.int32, device=DEV),
                            torch.zeros(1, dtype=torch.int32, device=DEV))
    lp = dsa.token_logprobs(logits, tok, 4)
    one, dx = torch.ones(26, device=DEV), torch.empty_like(logits)

    def step():
        k.copy_(k0), v.copy_(v0), w.copy_(w0)
        dsa.build_tree(c.cfg, parents, cu, out=bits, ws=ws[dsa.SERVE_WS_TREE])
        dsa.tree_attn(c.cfg, q, k, ptab, c.prefix, table, seq, cu, bits, v_pages=v, o=o, lse=lse,
                      ws=ws[dsa.SERVE_WS_PREFIX])
        dsa.key_weights(c.cfg, q, lse, k, table, seq, cu, w, tree_bits=bits,
                        ws=ws[dsa.SERVE_WS_WEIGHTS])
        dsa.evict_cache(c.cfg, w, table, seq, keep, k, v_pages=v, ws=ws[dsa.SERVE_WS_EVICT])
        dsa.release_pages(c.cfg, seq, keep, table, out=rel, ws=ws[dsa.SERVE_WS_TABLES])
        dsa.token_logprobs(logits, tok, 4, out=lp, ws=lws)
        dsa.token_logprobs_bwd(logits, tok, lp.lse, lp.entropy, one, one, dlogits=dx, ws=lws)

    results = lambda: [x.clone() for x in (bits, o, lse, w, k, v, *rel, *lp, dx)]
    step()
    torch.cuda.synchronize()
    want = results()
    assert head.shape[0] == 26 and rel.n_released.item() > 0
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for _ in range(4):
        for x in (o, lse, dx, *lp):
            x.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(results(), want))
    for x in (*ws.values(), lws):
        assert dsa.get_device_status(x) == 0


@gpu
def test_two_streams_at_once():
    """A workspace each; every result as the call alone gives it."""
    cases = [Case([6, 20], [100, 2300], 300, 16, 128, 16, 1, seed=s) for s in (5, 6)]
    evicts = [Evict([5000, 300, 20], [1000, 200, 30], 16, 128, 1, "few", seed=s) for s in (7, 8)]
    runs = []
    for c, e in zip(cases, evicts):
        dv = lambda t: t.to(DEV)
        bits = dv(signed(plain_bits(tree_parents(c.new, "random", 1), c.cu, 26, 1)))
        a = dict(c=c, e=e, q=dv(c.q), k=dv(torch.nan_to_num(c.k)), t=dv(c.table), s=i32(c.seq),
                 cu=i32(c.cu), bits=bits, lse=torch.full(c.q.shape[:2], 6.0, device=DEV),
                 w=torch.rand(c.k.shape[:2], device=DEV), ws=dsa.serve_workspace(
                     c.cfg, dsa.SERVE_WS_WEIGHTS, DEV), stream=torch.cuda.Stream(),
                 ew=dv(e.w), et=dv(e.table), el=i32(e.lens), ek=i32(e.keep),
                 ews=dsa.serve_workspace(e.cfg, dsa.SERVE_WS_EVICT, DEV), ec=dv(e.cache[0]))
        runs.append(a)

    def go(a):
        a["out"] = dsa.key_weights(a["c"].cfg, a["q"], a["lse"], a["k"], a["t"], a["s"], a["cu"],
                                   a["w"], tree_bits=a["bits"], w_out=torch.zeros_like(a["w"]),
                                   ws=a["ws"])
        cache = a["ec"].clone()
        w = dsa.evict_cache(a["e"].cfg, a["ew"], a["et"], a["el"], a["ek"], cache,
                            w_out=torch.zeros_like(a["ew"]), ws=a["ews"])
        return [a["out"], cache, w]

    want = [go(a) for a in runs]
    torch.cuda.synchronize()
    for _ in range(10):
        got = []
        for a in runs:
            with torch.cuda.stream(a["stream"]):
                got.append(go(a))
        torch.cuda.synchronize()
        for x, y in zip(got, want):
            assert all(torch.equal(p, r) for p, r in zip(x, y))
    for a in runs:
        assert dsa.get_device_status(a["ws"]) == dsa.get_device_status(a["ews"]) == 0


# ------------------------------------------- behind kernels that write late


@gpu
@pytest.mark.parametrize("captured", [False, True])
def test_calls_behind_a_kernel_that_writes_late(late, captured):  # noqa: F811
    c = Case([6, 20], [100, 230], 300, 16, 128, 16, 1, seed=13)
    dv = lambda t: t.to(DEV)
    bits = dv(signed(plain_bits(tree_parents(c.new, "random", 2), c.cu, 26, 1)))
    q, k, table, seq, cu = dv(c.q), dv(torch.nan_to_num(c.k)), dv(c.table), i32(c.seq), i32(c.cu)
    ptab, w = dv(c.prefix_table), torch.rand(c.k.shape[:2], device=DEV)
    ws = {x: dsa.serve_workspace(c.cfg, x, DEV) for x in (dsa.SERVE_WS_PREFIX, dsa.SERVE_WS_TREE,
                                                          dsa.SERVE_WS_WEIGHTS,
                                                          dsa.SERVE_WS_EVICT,
                                                          dsa.SERVE_WS_TABLES)}
    lws = dsa.logprobs_workspace(DEV)
    x, tok = logits_of(26, 4096, BF, 4)
    lse = dsa.tree_attn(c.cfg, q, k, ptab, c.prefix, table, seq, cu, bits,
                        ws=ws[dsa.SERVE_WS_PREFIX])[1]
    f = dsa.token_logprobs(x, tok, 3, ws=lws)
    keep, one = i32([60, 100]), torch.ones(26, device=DEV)
    parents = i32(tree_parents(c.new, "random", 2))
    o2, l2, t2 = torch.zeros_like(q), torch.zeros_like(lse), torch.zeros_like(bits)
    w2, k2, dx = torch.zeros_like(w), torch.zeros_like(k), torch.zeros_like(x)
    lp = dsa.TokenLogprobs(*[torch.zeros_like(a) for a in f])
    rel = dsa.ReleasedPages(*[torch.zeros(n, dtype=torch.int32, device=DEV) for n in (2, 30, 1)])

    def evict(a):
        k2.copy_(k)
        dsa.evict_cache(c.cfg, a, table, seq, keep, k2, w_out=w2, ws=ws[dsa.SERVE_WS_EVICT])
        return [k2, w2]

    calls = {
        "parents": (parents, lambda a: [dsa.build_tree(c.cfg, a, cu, out=t2,
                                                       ws=ws[dsa.SERVE_WS_TREE])]),
        "bits": (bits, lambda a: dsa.tree_attn(c.cfg, q, k, ptab, c.prefix, table, seq, cu, a, o=o2,
                                               lse=l2, ws=ws[dsa.SERVE_WS_PREFIX])),
        "lse": (lse, lambda a: [dsa.key_weights(c.cfg, q, a, k, table, seq, cu, w, tree_bits=bits,
                                                w_out=w2, ws=ws[dsa.SERVE_WS_WEIGHTS])]),
        "w": (w, lambda a: [dsa.key_weights(c.cfg, q, lse, k, table, seq, cu, a, w_out=w2,
                                            ws=ws[dsa.SERVE_WS_WEIGHTS])]),
        "rank": (w, evict),
        "seq": (seq, lambda a: dsa.release_pages(c.cfg, a, keep, table, out=rel,
                                                 ws=ws[dsa.SERVE_WS_TABLES])),
        "logits": (x, lambda a: dsa.token_logprobs(a, tok, 3, out=lp, ws=lws)),
        "g": (one, lambda a: [dsa.token_logprobs_bwd(x, tok, f.lse, f.entropy, a, dlogits=dx,
                                                     ws=lws)]),
    }
    for name, (value, call) in calls.items():
        have = value.clone()
        want = [a.clone() for a in call(have)]
        out = []

        def step():
            have.zero_()
            if name != "rank":
                late(have, value)
                out[:] = call(have)
            else:
                k2.copy_(k)
                late(have, value)
                dsa.evict_cache(c.cfg, have, table, seq, keep, k2, w_out=w2,
                                ws=ws[dsa.SERVE_WS_EVICT])
                out[:] = [k2, w2]

        replayed(step, captured)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, want)), name
    for a in (*ws.values(), lws):
        assert dsa.get_device_status(a) == 0


# --------------------------------------------------------- larger shapes


@gpu
@pytest.mark.parametrize("new,seq,H,words", [([300], [700], 16, 10), ([1000, 40], [1000, 40], 5, 32),
                                             ([70], [300], 16, 2)])
def test_large_trees(new, seq, H, words):
    """Nodes over several tiles; and more rows than the masks have nodes."""
    c = Case(new, seq, 100, H, 128, 64, 1, seed=sum(new))
    bits = plain_bits(tree_parents(new, "random", 7), c.cu, c.q.shape[0], words)
    check_tree(c, bits)
    weights_case(c, bits, 0.9, 3)


@gpu
def test_weights_of_many_requests():
    new = [(7 * b) % 23 for b in range(500)]
    seq = [n + (37 * b) % 300 for b, n in enumerate(new)]
    c = Case(new, seq, 0, 16, 128, 32, 1, seed=9)
    weights_case(c, plain_bits(tree_parents(new, "random", 9), c.cu, c.q.shape[0], 1), 0.5, 9)


@gpu
def test_caches_beyond_32_bit_offsets():
    """Pages whose elements lie past 2^31 of the cache."""
    page, d, n_pages = 128, 512, (1 << 31) // (128 * 512) + 200
    cfg = dsa.ServeConfig(n_pages=n_pages, max_tokens=2, batch=1, max_blocks=4, page_size=page,
                          attn_heads=16, d_qk=d, d_v=d)
    g = torch.Generator().manual_seed(1)
    k = torch.zeros((n_pages, page, d), dtype=BF, device=DEV)
    ids = [n_pages - 1, 3, n_pages - 57, n_pages - 2]
    rows = torch.randn((4, page, d), generator=g).to(BF)
    k[torch.tensor(ids, device=DEV)] = rows.to(DEV)
    q = torch.randn((2, 16, d), generator=g).to(BF)
    small = types.SimpleNamespace(q=q, k=rows, v=rows, prefix=0, seq=[400], cu=[0, 2],
                                  prefix_table=torch.zeros(0, dtype=torch.int32),
                                  table=torch.arange(4, dtype=torch.int32)[None], cfg=cfg)
    bits = [[1], [2]]
    table, seq, cu = i32([ids]), i32([400]), i32([0, 2])
    o, lse = dsa.tree_attn(cfg, q.to(DEV), k, None, 0, table, seq, cu, signed(bits).to(DEV))
    check([o.cpu(), lse.cpu()], plain_tree(small, bits))
    w = torch.rand((n_pages, page), generator=g)
    got = dsa.key_weights(cfg, q.to(DEV), lse, k, table, seq, cu, w.to(DEV),
                          tree_bits=signed(bits).to(DEV)).cpu()
    want, tol = plain_weights(small, bits, lse.cpu(), w[ids], w[ids], 1.0)
    assert ((got[ids].double().view(-1) - want).abs() <= tol).all()
    dsa.evict_cache(cfg, got.to(DEV), table, seq, i32([130]), k)
    src = plain_keep(got[ids].view(-1)[:400].tolist(), 130, 0, 0)
    assert torch.equal(k[torch.tensor(ids, device=DEV)].cpu().view(-1, d)[:130],
                       rows.view(-1, d)[src])


# ---------------------------------------------------------- checks build


CHILD = """
import json, torch
import long_context_sparse_gb300 as dsa
from tests.test_evict import Evict
from tests.test_logprobs import check as logp, check_grad, logits_of
from tests.test_serving import Case, DEV
from tests.test_tree import check_tree, plain_bits, tree_parents, weights_case
c = Case([30, 0, 7], [300, 20, 7], 700, 16, 256, 64, 2, seed=5)
bits = plain_bits(tree_parents(c.new, "random", 1), c.cu, 37, 1)
check_tree(c, bits)
weights_case(c, bits, 0.9, 1)
from tests.test_evict import check_evict
check_evict(Evict([9000, 300, 7], [2000, 100, 9], 16, 128, 2, "few", seed=1), n_last=5)
x, tok = logits_of(40, 50001, torch.bfloat16, 1)
logp(x, tok, 20, 1.0)
check_grad(x, tok, 1.0, 1)
print(json.dumps(dsa.library_path()))
"""


@gpu
def test_the_checks_build_agrees():
    r = subprocess.run([sys.executable, "-c", CHILD], capture_output=True, text=True, timeout=600,
                       env=dict(os.environ, DSA_GB300_CHECKS="1"))
    assert r.returncode == 0, r.stderr[-2000:]
    assert json.loads(r.stdout.strip().splitlines()[-1]).endswith("libdsa_gb300_checks.so")
