"""Serving calls side by side: captured graphs replayed at once on two streams,
steps on two streams, and pages that several lists hold."""
import pytest
import torch

import long_context_sparse_gb300 as dsa
from tests.test_serving import BF, DEV, Case, check, check_case, plain_attn

gpu = pytest.mark.gpu


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


@gpu
def test_two_graphs_replayed_at_once():
    """A workspace each; every result as the call alone gives it, bit for bit."""
    cases = [Case([1, 2], [40, 300], 30000, 16, 512, 64, 1, seed=61),
             Case([1] * 40, [33] * 40, 2000, 64, 256, 32, 2, seed=62)]
    graphs, outs, refs, keep, spaces = [], [], [], [], []
    for c in cases:
        refs.append(c.run())
        args = [x.to(DEV) for x in (c.q, c.k, c.prefix_table)]
        rest = [c.table.to(DEV), i32(c.seq), i32(c.cu)]
        v = c.v.to(DEV) if c.kv == 2 else None
        o = torch.zeros(c.q.shape, dtype=BF, device=DEV)
        lse = torch.zeros(c.q.shape[:2], device=DEV)
        ws = dsa.serve_workspace(c.cfg, dsa.SERVE_WS_PREFIX, DEV)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            for _ in range(3):
                dsa.prefix_attn(c.cfg, *args, c.prefix, *rest, v_pages=v, o=o, lse=lse, ws=ws)
        graphs.append(g), outs.append((o, lse)), keep.append((args, rest, v)), spaces.append(ws)
    streams = [torch.cuda.Stream() for _ in cases]
    for _ in range(20):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for (o, lse), ref, ws in zip(outs, refs, spaces):
        assert dsa.get_device_status(ws) == 0
        assert torch.equal(o.cpu(), ref[0]) and torch.equal(lse.cpu(), ref[1])


@gpu
def test_steps_of_two_engines_at_once():
    """Tables, append and attention of two caches, a stream and workspaces each,
    call by call in turn."""
    B, H, P, page, d, n_pages, width, T = 3, 16, 300, 32, 128, 60, 10, 20
    cfg = dsa.ServeConfig(n_pages=n_pages, max_tokens=T, batch=B, max_blocks=width,
                          page_size=page, attn_heads=H, d_qk=d, d_v=d)
    g = torch.Generator().manual_seed(5)
    bf = lambda *s: torch.randn(s, generator=g).to(BF).to(DEV)
    engines = []
    for e in range(2):
        engines.append(dict(
            s=torch.cuda.Stream(), k=bf(n_pages, page, d), q=bf(T, H, d), rows=bf(T, d),
            ptab=i32(list(range(10))), free=i32(list(range(59, 9, -1))),
            table=torch.full((B, width), -1, dtype=torch.int32, device=DEV),
            lens=i32([0] * B), new=i32([4 + e, 0, 11 - e]),
            ws=[dsa.serve_workspace(cfg, w, DEV) for w in range(3)]))
    torch.cuda.synchronize()
    for _ in range(5):
        for e in engines:
            with torch.cuda.stream(e["s"]):
                e["t"] = dsa.build_page_tables(cfg, e["lens"], e["new"], e["free"], e["table"],
                                               ws=e["ws"][0])
        for e in engines:
            with torch.cuda.stream(e["s"]):
                dsa.append_cache(cfg, e["t"].slot_map, e["rows"], e["k"], ws=e["ws"][1])
        for e in engines:
            with torch.cuda.stream(e["s"]):
                e["o"] = dsa.prefix_attn(cfg, e["q"], e["k"], e["ptab"], P, e["table"],
                                         e["t"].seq_lens, e["t"].cu_tokens, ws=e["ws"][2])
    torch.cuda.synchronize()
    for e in engines:
        assert [dsa.get_device_status(w) for w in e["ws"]] == [0, 0, 0]
        cu, slots = e["t"].cu_tokens.tolist(), e["t"].slot_map.tolist()
        for x in range(cu[-1]):
            assert torch.equal(e["k"].view(-1, d)[slots[x]], e["rows"][x])
        k = e["k"].cpu()
        check([x.cpu() for x in e["o"]],
              plain_attn(e["q"].cpu(), k, k, e["ptab"].cpu(), P, e["table"].cpu(),
                         e["t"].seq_lens.tolist(), cu, cfg.scale))


@gpu
def test_pages_in_several_lists_and_twice_in_one():
    """What is only read may be listed anywhere: a page of the prefix twice in it
    and in a request's table, two requests with one page."""
    c = Case([1, 3, 1], [64, 130, 64], 600, 16, 256, 64, 2, seed=63)
    c.prefix_table[3] = c.prefix_table[0]
    c.prefix_table[5] = c.prefix_table[0]
    c.table[1, 0] = c.prefix_table[1]
    c.table[2, 0] = c.table[0, 0]
    check_case(c)
