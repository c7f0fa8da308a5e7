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
