"""Offsets of the rows that are out of order in ways that 32-bit differences and
products hide: the calls say so, and read and write nothing."""
import pytest
import torch

import long_context_sparse_gb300 as dsa
from tests.test_serving import BF, DEV
from tests.test_tree import i32

gpu = pytest.mark.gpu

# (H, T, cu_tokens).  A difference times the heads, or a difference alone, passes
# 2^32 and comes out as a number of rows that could be.
WRAPPED = [
    (16, 8, [0, 100000000, 200000000, 268435456, 8]),  # products: 1.6e9, 1.6e9, 1.1e9, 128 rows
    (16, 8, [0, 1 << 28, 4]),                          # 0 and 64 rows
    (64, 1000, [0, 33554431, 67108862, 1000]),
    (1, 8, [0, (1 << 31) - 1, -2, 5]),                 # differences: 2^31 - 1, 2^31 - 1, 7
    (16, 8, [0, (1 << 31) - 1, -2, 5]),
    (128, 8, [0, 1 << 25, 8]),
]


def wraps(x):
    return (x + (1 << 31)) % (1 << 32) - (1 << 31)


def test_the_offsets_pass_where_only_signs_are_looked_at():
    """Each of them from 0 to at most T, out of order, with no negative number of rows by
    32-bit products or by 32-bit differences."""
    for H, T, cu in WRAPPED:
        assert cu[0] == 0 and cu[-1] <= T
        assert any(a > b for a, b in zip(cu, cu[1:]))
        gaps = [wraps(b - a) for a, b in zip(cu, cu[1:])]
        assert min(gaps) >= 0 or min(wraps(n * H) for n in gaps) >= 0


def requests(H, T, cu, spread):
    """A small cache for the offsets; `spread`: more requests than a warp has lanes."""
    if spread:
        cu = cu[:2] + [cu[1]] * 700 + cu[2:]
    B = len(cu) - 1
    cfg = dsa.ServeConfig(n_pages=16, max_tokens=T, batch=B, max_blocks=2, page_size=16,
                          attn_heads=H, d_qk=128, d_v=128)
    g = torch.Generator().manual_seed(H + T)
    k = torch.randn((16, 16, 128), generator=g).to(BF).to(DEV)
    q = torch.randn((T, H, 128), generator=g).to(BF).to(DEV)
    table = (torch.arange(2 * B, dtype=torch.int32) % 16).view(B, 2).to(DEV)
    return cfg, k, q, table, i32([20] * B), i32(cu)


@gpu
@pytest.mark.parametrize("spread", [False, True])
@pytest.mark.parametrize("H,T,cu", WRAPPED)
def test_weights_latch_offsets_that_wrap(H, T, cu, spread):
    cfg, k, q, table, seq, cu = requests(H, T, cu, spread)
    ws = dsa.serve_workspace(cfg, dsa.SERVE_WS_WEIGHTS, DEV)
    w = torch.rand((16, 16), device=DEV)
    for bits in (None, torch.full((T, 1), -1, dtype=torch.int32, device=DEV)):
        out = dsa.key_weights(cfg, q, torch.zeros((T, H), device=DEV), k, table, seq, cu, w,
                              tree_bits=bits, w_out=torch.full_like(w, 7.0), ws=ws)
        assert dsa.get_device_status(ws) == 7
        assert (out == 7.0).all()


@gpu
@pytest.mark.parametrize("spread", [False, True])
@pytest.mark.parametrize("H,T,cu", WRAPPED)
def test_attention_latches_offsets_that_wrap(H, T, cu, spread):
    """By trees and in order, with a prefix and without: nothing behind the results or the
    workspace is written."""
    cfg, k, q, table, seq, cu = requests(H, T, cu, spread)
    need = dsa.serve_workspace_size(cfg, dsa.SERVE_WS_PREFIX)
    for prefix in (0, 40):
        for bits in (None, torch.full((T, 1), -1, dtype=torch.int32, device=DEV)):
            ws = torch.zeros(need + 4096, dtype=torch.uint8, device=DEV)
            ws[need:] = 85
            o = torch.full((T + 8, H, 128), 7.0, dtype=BF, device=DEV)
            lse = torch.full((T + 8, H), 7.0, device=DEV)
            args = (cfg, q, k, i32([3, 4, 5]), prefix, table, seq, cu)
            out = dict(o=o[:T], lse=lse[:T], ws=ws)
            if bits is None:
                dsa.prefix_attn(*args, **out)
            else:
                dsa.tree_attn(*args, bits, **out)
            assert dsa.get_device_status(ws) == 7
            assert (o[T:] == 7.0).all() and (lse[T:] == 7.0).all() and (ws[need:] == 85).all()
