"""Evictions one after the other: what an earlier call left behind does not reach a later
one."""
import pytest
import torch

import long_context_sparse_gb300 as dsa
from tests.test_evict import Evict
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
