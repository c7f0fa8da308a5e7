"""Attention for trees of drafted tokens, and the weights that cached tokens
receive, against plain definitions (masks by walking up, products in fp64)."""
import ctypes
import math

import numpy as np
import pytest
import torch

import long_context_sparse_gb300 as dsa
from long_context_sparse_gb300 import build as dsa_build
from tests.test_serving import BF, DEV, Case, check

gpu = pytest.mark.gpu
P = ctypes.c_void_p


def i32(x, dev=DEV):
    return torch.tensor(x, dtype=torch.int32, device=dev)


# ----------------------------------------------------- plain definitions


def plain_bits(parents, cu, T, words):
    """[T, words] of Python integers, bit j % 32 of word j / 32: node j is seen."""
    bits = [[0] * words for _ in range(T)]
    for b in range(len(cu) - 1):
        for i in range(cu[b + 1] - cu[b]):
            j = i
            while j >= 0:
                if j < 32 * words:
                    bits[cu[b] + i][j // 32] |= 1 << (j % 32)
                j = parents[cu[b] + j]
    return bits


def signed(bits):
    return torch.tensor([[x - (1 << 32) if x >> 31 else x for x in r] for r in bits],
                        dtype=torch.int32).view(len(bits), -1)


def tree_parents(new, kind, seed):
    """Parents of every row: random trees, chains, stars or roots only."""
    g = torch.Generator().manual_seed(seed)
    out = []
    for n in new:
        for i in range(n):
            up = {"chain": i - 1, "star": min(0, i - 1), "roots": -1}.get(kind)
            out.append(int(torch.randint(-1, i, (1,), generator=g)) if up is None else up)
    return out


def seen_own(bits, base, n, rows, first):
    """[rows, n]: which own tokens the rows from `first` on see."""
    see = torch.zeros(rows, n, dtype=torch.bool)
    for i in range(rows):
        for pos in range(n):
            j = pos - base
            see[i, pos] = j < 0 or (j < 32 * len(bits[first + i]) and
                                    bits[first + i][j // 32] >> (j % 32) & 1)
    return see


def plain_tree(c, bits):
    """fp64 (O, LSE, sum_j P_j |v_j|) as plain_attn of the serving tests, by tree."""
    T, H, d = c.q.shape
    page = c.k.shape[1]
    o = torch.full((T, H, d), math.nan, dtype=torch.float64)
    mag, lse = o.clone(), torch.full((T, H), math.nan, dtype=torch.float64)
    rows = lambda x, pages, n: x[pages[: -(-n // page)].long()].reshape(-1, d)[:n].double()
    kp, vp = (rows(x, c.prefix_table, c.prefix) for x in (c.k, c.v))
    for b, n in enumerate(c.seq):
        lo, hi = c.cu[b], c.cu[b + 1]
        if lo == hi:
            continue
        kk = torch.cat([kp, rows(c.k, c.table[b], n)])
        vv = torch.cat([vp, rows(c.v, c.table[b], n)])
        s = torch.einsum("ihd,jd->ihj", c.q[lo:hi].double(), kk) * c.cfg.scale
        see = torch.cat([torch.ones(hi - lo, c.prefix, dtype=torch.bool),
                         seen_own(bits, n - (hi - lo), n, hi - lo, lo)], 1)
        s = s.masked_fill(~see[:, None, :], -math.inf)
        p = torch.softmax(s, -1).nan_to_num(0.0) if kk.shape[0] else s
        o[lo:hi], mag[lo:hi] = p @ vv, p @ vv.abs()
        lse[lo:hi] = torch.logsumexp(s, -1)
    return o, lse, mag


def run_tree(c, bits, ws=None, o=None, lse=None):
    dv = lambda t: t.to(DEV)
    kd = dv(c.k)
    ws = dsa.serve_workspace(c.cfg, dsa.SERVE_WS_PREFIX, DEV) if ws is None else ws
    o, lse = dsa.tree_attn(c.cfg, dv(c.q), kd, dv(c.prefix_table), c.prefix, dv(c.table),
                           i32(c.seq), i32(c.cu), dv(bits),
                           v_pages=None if c.kv == 1 else dv(c.v), o=o, lse=lse, ws=ws)
    torch.cuda.synchronize()
    return o.cpu(), lse.cpu(), dsa.get_device_status(ws)


def check_tree(c, bits):
    *got, status = run_tree(c, signed(bits))
    assert status == 0
    check(got, plain_tree(c, bits))
    return got


# ------------------------------------------------------------ host checks


@pytest.fixture(scope="module")
def lib():
    dsa_build.build()
    return dsa._load()


def scfg(**kw):
    base = dict(n_pages=100, max_tokens=8, batch=4, max_blocks=10, page_size=64, attn_heads=16,
                d_qk=128, d_v=128)
    base.update(kw)
    return dsa.ServeConfig(**base)


def refusals(call, size, written, ok_pairs=()):
    """Every written buffer on every other, at its start and at its end: refused."""
    at = {n: (i + 1) << 28 for i, n in enumerate(size)}
    assert max(size.values()) < 1 << 28
    for w in written:
        step = 256 if w == "ws" else 16
        for x in size:
            if x == w or (w, x) in ok_pairs:
                continue
            assert call(at, **{w: at[x]}) == 1, (w, x)
            assert call(at, **{w: at[x] + (size[x] - 1) // step * step}) == 1, (w, x)
            assert call(at, **{x: at[w] + (size[w] - 1) // 256 * 256}) == 1, (w, x)


def test_build_tree_refusals(lib):
    c = scfg()
    r = ctypes.byref(c.c())
    p, q, o, ws = P(256), P(1024), P(2048), P(4096)
    f = lib.dsa_build_tree
    assert f(r, p, q, 0, o, ws, 256, None) == 1
    assert f(r, p, q, 33, o, ws, 256, None) == 1
    assert f(r, None, q, 1, o, ws, 256, None) == 1
    assert f(r, p, q, 1, P(2052), ws, 256, None) == 4
    assert f(r, p, q, 1, o, ws, 255, None) == 3
    assert f(r, p, q, 1, o, P(4100), 256, None) == 4
    size = dict(parents=32, cu=20, bits=8 * 3 * 4, ws=256)

    def call(at, **over):
        a = {**at, **over}
        return f(r, P(a["parents"]), P(a["cu"]), 3, P(a["bits"]), P(a["ws"]), 256, None)

    refusals(call, size, ("bits", "ws"))


def test_tree_attn_refusals(lib):
    T, H, B, d, page, words = 8, 16, 4, 128, 64, 2
    c = scfg()
    r = ctypes.byref(c.c())
    nb = dsa.serve_workspace_size(c, dsa.SERVE_WS_PREFIX)
    f = lib.dsa_tree_attn
    size = dict(q=T * H * d * 2, k=100 * page * d * 2, v=100 * page * d * 2, prefix=16,
                table=B * 40, seq=B * 4, cu=B * 4 + 4, bits=T * words * 4, o=T * H * d * 2,
                lse=T * H * 4, ws=nb)

    def call(at, words=words, ws_bytes=nb, **over):
        q, k, v, pt, table, seq, cu, bits, o, lse, ws = (P(x) for x in {**at, **over}.values())
        return f(r, q, k, v, pt, 200, table, seq, cu, bits, words, o, lse, ws, ws_bytes, None)

    refusals(call, size, ("o", "lse", "ws"), (("o", "q"), ("lse", "q")))
    at = {n: (i + 1) << 28 for i, n in enumerate(size)}
    assert call(at, bits=None) == 1 and call(at, words=0) == 1 and call(at, words=33) == 1
    assert call(at, bits=at["bits"] + 4) == 4 and call(at, ws_bytes=nb - 1) == 3
    big = scfg(max_tokens=1 << 17)
    r = ctypes.byref(big.c())
    assert call(at) == 2


def test_key_weights_refusals(lib):
    T, H, B, d, page, words = 8, 16, 4, 128, 64, 2
    c = scfg()
    r = ctypes.byref(c.c())
    nb = dsa.serve_workspace_size(c, dsa.SERVE_WS_WEIGHTS)
    f = lib.dsa_key_weights
    size = dict(q=T * H * d * 2, lse=T * H * 4, k=100 * page * d * 2, table=B * 40, seq=B * 4,
                cu=B * 4 + 4, bits=T * words * 4, w=100 * page * 4, out=100 * page * 4, ws=nb)

    def call(at, words=words, decay=0.5, ws_bytes=nb, **over):
        q, lse, k, table, seq, cu, bits, w, out, ws = (P(x) for x in {**at, **over}.values())
        return f(r, q, lse, k, table, seq, cu, bits, words, w, decay, out, ws, ws_bytes, None)

    at = {n: (i + 1) << 28 for i, n in enumerate(size)}
    for x in size:
        if x not in ("out", "w"):
            assert call(at, out=at[x]) == 1, x
        if x != "ws":
            assert call(at, ws=at[x]) == 1, x
    assert call(at, out=at["w"] + 256) == 1            # in place means in the same place
    assert call(at, w=None) == 1 and call(at, words=0) == 1
    for decay in (-0.1, 1.5, math.nan):
        assert call(at, decay=decay) == 1
    assert call(at, lse=at["lse"] + 4) == 4
    assert call(at, ws_bytes=nb - 1) == 3
    with pytest.raises(dsa.DsaError) as e:
        dsa.serve_workspace_size(scfg(max_tokens=1 << 17), dsa.SERVE_WS_WEIGHTS)
    assert e.value.code == 2


def test_workspaces_of_the_tree_calls(lib):
    big = scfg(max_tokens=1 << 20, attn_heads=1000, d_qk=96, d_v=96)  # heads do not matter
    assert dsa.serve_workspace_size(big, dsa.SERVE_WS_TREE) == 256
    for which in (15, 19):
        with pytest.raises(dsa.DsaError) as e:
            dsa.serve_workspace_size(scfg(), which)
        assert e.value.code == 1


def test_python_refuses_wrong_tree_tensors():
    c, i = scfg(), torch.zeros(8, dtype=torch.int32)
    with pytest.raises(ValueError):       # not on a GPU
        dsa.build_tree(c, i, torch.zeros(5, dtype=torch.int32))
    with pytest.raises(ValueError):
        dsa.tree_attn(c, None, None, None, 0, None, None, None, None)
    with pytest.raises(TypeError):
        dsa.key_weights(c, None, None, None, None, None, None, None)


# ----------------------------------------------------------------- masks


@gpu
@pytest.mark.parametrize("new,words,kind", [
    ([1], 1, "random"), ([0, 3, 0, 32, 33, 64], 2, "random"), ([64] * 5, 2, "chain"),
    ([1024, 7], 32, "random"), ([1000], 32, "chain"), ([100, 31], 4, "star"),
    ([5, 40], 2, "roots"), ([17] * 700, 1, "random")])
def test_build_tree(new, words, kind):
    T = sum(new) + 3
    parents = tree_parents(new, kind, len(new)) + [77, -5, 0]
    cu = [0]
    for n in new:
        cu.append(cu[-1] + n)
    cfg = scfg(max_tokens=T, batch=len(new))
    ws = dsa.serve_workspace(cfg, dsa.SERVE_WS_TREE, DEV)
    out = torch.full((T, words), 99, dtype=torch.int32, device=DEV)
    got = dsa.build_tree(cfg, i32(parents), i32(cu), out=out, ws=ws)
    assert got is out and dsa.get_device_status(ws) == 0
    assert torch.equal(out[: T - 3].cpu(), signed(plain_bits(parents, cu, T - 3, words)))
    assert (out[T - 3:] == 99).all()      # rows of no request


@gpu
def test_build_tree_latches_what_is_wrong():
    for parents, cu, words in (([0, 0], [0, 2], 1), ([-2, 0], [0, 2], 1), ([-1, 1], [0, 2], 1),
                               ([-1] * 40, [0, 40], 1), ([-1, 0], [0, 3], 1),
                               ([-1, 0], [2, 0], 1), ([-1, 0], [-1, 1], 1)):
        cfg = scfg(max_tokens=len(parents), batch=1)
        ws = dsa.serve_workspace(cfg, dsa.SERVE_WS_TREE, DEV)
        out = dsa.build_tree(cfg, i32(parents), i32(cu), words=words, ws=ws)
        assert dsa.get_device_status(ws) == 7, (parents, cu)
        if len(parents) == 40:            # more nodes than bits: nothing is written
            assert (out == 0).all()
        if cu == [0, 2]:                  # taken for a root
            assert out[1, 0].item() in (2, 3) and out[0, 0].item() == 1
    # a request without soundness leaves the others alone
    cfg = scfg(max_tokens=4, batch=2)
    ws = dsa.serve_workspace(cfg, dsa.SERVE_WS_TREE, DEV)
    out = dsa.build_tree(cfg, i32([-1, 0, -1, 0]), i32([0, 2, 9]), words=1, ws=ws)
    assert dsa.get_device_status(ws) == 7 and out[:, 0].tolist() == [1, 3, 0, 0]


# ------------------------------------------------------------- attention


CASES = [
    # new, own tokens, prefix, H, d, page, kv
    ([1], [1], 0, 1, 128, 16, 1),
    ([7], [7], 0, 16, 512, 64, 1),                 # nodes alone
    ([7], [40], 1021, 16, 512, 64, 1),
    ([64], [64], 0, 1, 128, 16, 2),                # 64 nodes in a group of rows
    ([100, 64], [400, 65], 30, 1, 256, 32, 2),     # one head: more nodes than a group has
    ([33, 0, 5], [300, 77, 261], 500, 3, 256, 32, 2),
    ([20, 31], [255, 256 + 31], 0, 5, 128, 16, 1),  # nodes on both sides of a tile's end
    ([9, 40, 1], [9 + 256, 300, 512], 257, 64, 512, 128, 2),
    ([12, 3], [500, 3], 100, 128, 128, 64, 1),
    ([64] * 3, [64 + 31, 64 + 32, 64 + 33], 0, 8, 128, 16, 2),
    ([2, 5], [1, 2], 300, 16, 256, 64, 2),         # fewer own tokens than rows
    ([30], [5000], 3000, 24, 512, 64, 1),
]


@gpu
@pytest.mark.parametrize("i", range(len(CASES)))
@pytest.mark.parametrize("kind", ["random", "star", "roots"])
def test_tree_attention(i, kind):
    new, seq, prefix, H, d, page, kv = CASES[i]
    c = Case(new, seq, prefix, H, d, page, kv, pad=2, seed=100 + i, extra=1)
    words = -(-max(new) // 32)
    bits = plain_bits(tree_parents(new, kind, i) + [0, 0], c.cu, c.q.shape[0], words)
    check_tree(c, bits)


@gpu
@pytest.mark.parametrize("i", [1, 4, 5, 6, 9])
def test_bits_of_any_kind(i):
    """Masks that no tree makes: any nodes, none at all, nodes that come later; rows
    that see nothing but the prefix, or nothing."""
    new, seq, prefix, H, d, page, kv = CASES[i]
    c = Case(new, seq, prefix, H, d, page, kv, seed=200 + i)
    g = torch.Generator().manual_seed(i)
    words = -(-max(new) // 32) + 1
    bits = torch.randint(0, 1 << 32, (c.q.shape[0], words), generator=g)
    bits[::3] = 0
    got = check_tree(c, bits.tolist())
    if prefix == 0 and new == seq:
        assert (got[0][0] == 0).all() and torch.isinf(got[1][0]).all()


@gpu
def test_a_chain_is_the_prefix_attention():
    c = Case([30, 1, 64], [300, 1, 700], 900, 16, 256, 64, 2, seed=7)
    bits = signed(plain_bits(tree_parents(c.new, "chain", 0), c.cu, c.q.shape[0], 2))
    o, lse, status = run_tree(c, bits)
    ref = c.run()
    assert status == ref[2] == 0
    # equal sums in another order of references: one rounding of O each way, fp32 in LSE
    assert (o.double() - ref[0].double()).abs().max() <= 2.0 ** -7 * ref[0].double().abs().max()
    assert (lse - ref[1]).abs().max() <= 2.0 ** -18 * ref[1].abs().max()


@gpu
def test_scores_that_raise_references_among_the_nodes():
    """Each later node scores far above those before it, in other orders for other
    rows: references are raised, and first set, inside the tile of the nodes."""
    for base in (0, 40, 256):
        c = Case([50], [50 + base], 0, 16, 128, 16, 2, seed=base + 1, qscale=1.0)
        c.q = torch.ones_like(c.q)
        k = c.k.view(-1, 128)
        for pos in range(50 + base):
            slot = int(c.table[0, pos // 16]) * 16 + pos % 16
            k[slot] = 0.01 * (pos % 5) if pos < base else 0.25 * (pos - base) - 3.0
        bits = plain_bits(tree_parents([50], "random", base), c.cu, 50, 2)
        check_tree(c, bits)
        full = [[0xFFFFFFFF, 0xFFFFFFFF]] * 50
        check_tree(c, full)
        none_but_last = [[0, 1 << 17]] * 50       # node 49, beyond the first 32 keys
        check_tree(c, none_but_last)


@gpu
def test_many_requests_and_items():
    new = [(7 * b) % 23 for b in range(300)]
    seq = [n + (37 * b) % 500 for b, n in enumerate(new)]
    c = Case(new, seq, 600, 16, 128, 32, 2, seed=9)
    bits = plain_bits(tree_parents(new, "random", 9), c.cu, c.q.shape[0], 1)
    check_tree(c, bits)


@gpu
def test_masked_nodes_do_not_reach_others_and_results_repeat():
    """K of a node that no row sees may be infinite or NaN; every replay of a graph
    gives the same bits."""
    c = Case([10], [70], 300, 16, 128, 16, 2, seed=11)
    bits = plain_bits(tree_parents([10], "random", 3), c.cu, 10, 1)
    bits = [[x & ~(1 << 4)] for (x,) in bits]
    want = plain_tree(c, bits)
    slot = int(c.table[0, 64 // 16]) * 16
    k = c.k.clone()
    k.view(-1, 128)[slot] = math.nan
    c.k = k
    *got, status = run_tree(c, signed(bits))
    assert status == 0
    check(got, want)
    ws = dsa.serve_workspace(c.cfg, dsa.SERVE_WS_PREFIX, DEV)
    args = [x.to(DEV) for x in (c.q, c.k, c.prefix_table)]
    rest = [c.table.to(DEV), i32(c.seq), i32(c.cu), signed(bits).to(DEV)]
    o, lse = torch.zeros_like(args[0]), torch.zeros(args[0].shape[:2], device=DEV)
    v = c.v.to(DEV)
    call = lambda: dsa.tree_attn(c.cfg, *args, c.prefix, *rest, v_pages=v, o=o, lse=lse, ws=ws)
    call()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    for _ in range(3):
        o.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(o.cpu(), got[0]) and torch.equal(lse.cpu(), got[1])


# --------------------------------------------------------------- weights


def plain_weights(c, bits, lse, w, out, decay):
    """fp64 (w_out, bound on its error) for fp32 lse and w."""
    H, d = c.q.shape[1:]
    page = c.k.shape[1]
    out, tol = out.double().clone().view(-1), torch.zeros(out.numel(), dtype=torch.float64)
    w = w.view(-1)
    for b, n in enumerate(c.seq):
        lo, hi = c.cu[b], c.cu[b + 1]
        if lo == hi:
            continue
        rows, base = hi - lo, n - (hi - lo)
        slots = torch.tensor([int(c.table[b, p // page]) * page + p % page for p in range(n)],
                             dtype=torch.long)
        kk = c.k.view(-1, d)[slots].double()
        q = c.q[lo:hi].double()
        s = torch.einsum("ihd,jd->ihj", q, kk) * c.cfg.scale
        size = torch.einsum("ihd,jd->ihj", q.abs(), kk.abs()) * c.cfg.scale
        if bits is None:
            see = torch.arange(n)[None, :] <= (base + torch.arange(rows))[:, None]
        else:
            see = seen_own(bits, base, n, rows, lo)
        x = lse[lo:hi].double()[..., None]
        p = torch.where(see[:, None, :] & (x > -math.inf), torch.exp(s - x), 0.0)
        # a sum of d products errs by d 2^-24 of their sizes; the exponent's own
        # roundings by 2^-22 of it; the sum of rows * H terms by that many 2^-24
        err = p * (d * 2.0 ** -24 * size + 2.0 ** -22 * ((s - x).abs().clamp(max=200) + 2)
                   + rows * H * 2.0 ** -24)
        old = torch.where(torch.arange(n) < base, decay * w[slots].double(), 0.0)
        out[slots] = old + p.sum((0, 1))
        tol[slots] = torch.nan_to_num(err).sum((0, 1)) + 2.0 ** -22 * old.abs()
    return out, tol + 1e-37


def weights_case(c, bits, decay, seed, in_place=False):
    g = torch.Generator().manual_seed(seed)
    if bits is not None:
        lse = plain_tree(c, bits)[1]
    else:
        lse = c.plain()[1]
    lse = torch.nan_to_num(lse, nan=5.0, neginf=-math.inf).float()
    w = torch.rand(c.k.shape[:2], generator=g)
    out = w if in_place else torch.full_like(w, 7.0)
    want, tol = plain_weights(c, bits, lse, w, out, decay)
    ws = dsa.serve_workspace(c.cfg, dsa.SERVE_WS_WEIGHTS, DEV)
    wd = w.to(DEV)
    od = wd if in_place else out.to(DEV)
    got = dsa.key_weights(c.cfg, c.q.to(DEV), lse.to(DEV), c.k.to(DEV), c.table.to(DEV),
                          i32(c.seq), i32(c.cu), wd,
                          tree_bits=None if bits is None else signed(bits).to(DEV), decay=decay,
                          w_out=od, ws=ws)
    assert dsa.get_device_status(ws) == 0
    err = (got.cpu().double().view(-1) - want).abs() - tol
    assert (err <= 0).all(), f"{err.max():.3g} over the bound"
    return got.cpu()


@gpu
@pytest.mark.parametrize("i", range(len(CASES)))
@pytest.mark.parametrize("tree", [False, True])
def test_key_weights(i, tree):
    new, seq, prefix, H, d, page, kv = CASES[i]
    c = Case(new, seq, prefix, H, d, page, kv, pad=2, seed=300 + i, extra=1)
    bits = None
    if tree:
        words = -(-max(new) // 32)
        bits = plain_bits(tree_parents(new, "random", i) + [0, 0], c.cu, c.q.shape[0], words)
    weights_case(c, bits, 0.75 if i % 2 else 1.0, i, in_place=i % 3 == 0)


@gpu
@pytest.mark.parametrize("T,n,H,d", [(1, 4000, 64, 512), (200, 700, 16, 512), (130, 129, 128, 128),
                                     (300, 1000, 5, 256)])
def test_weights_of_many_rows_and_keys(T, n, H, d):
    c = Case([T, 1], [n, 300], 0, H, d, 64, 1, seed=T)
    weights_case(c, None, 0.9, T)


@gpu
def test_weights_of_any_bits_and_of_rows_without_keys():
    c = Case([40, 3], [40, 3], 0, 8, 128, 16, 1, seed=31)
    g = torch.Generator().manual_seed(1)
    bits = torch.randint(0, 1 << 32, (43, 2), generator=g)
    bits[::2] = 0                                   # lse = -inf: nothing is added
    got = weights_case(c, bits.tolist(), 1.0, 5)
    assert torch.isfinite(got).all()


@gpu
def test_weights_sum_to_the_rows():
    """Without a prefix, every row gives its tokens 1 in all."""
    c = Case([3, 20], [500, 20], 0, 16, 256, 32, 1, seed=41)
    out = torch.zeros(c.k.shape[:2])
    got = weights_case(c, None, 0.0, 3)
    for b in range(2):
        n = c.seq[b]
        slots = [int(c.table[b, p // 32]) * 32 + p % 32 for p in range(n)]
        assert abs(got.view(-1)[slots].double().sum() - 16 * c.new[b]) < 16 * c.new[b] * 2e-3
    assert out.shape == got.shape


@gpu
@pytest.mark.parametrize("d,page", [(128, 16), (256, 64), (512, 16), (512, 128)])
def test_weights_of_many_short_requests(d, page):
    """Several units a pair, with rows of all sizes behind one another; and one request's
    NaN stays with it, whatever the others' tiles find in its place."""
    rng = np.random.default_rng(d + page)
    B = 330
    new = [int(x) for x in rng.choice([0, 1, 1, 2, 4, 9, 30], B)]
    seq = [max(n, int(x)) for n, x in zip(new, rng.integers(1, 300, B))]
    new[7], seq[7] = 3, 200
    c = Case(new, seq, 0, 16, d, page, 1, seed=d)
    clean = weights_case(c, None, 0.5, 9)
    lse = torch.nan_to_num(c.plain()[1], nan=5.0, neginf=-math.inf).float().to(DEV)
    w = torch.rand(c.k.shape[:2], generator=torch.Generator().manual_seed(9)).to(DEV)
    k = c.k.clone()
    mine = torch.zeros(c.k.shape[:2], dtype=torch.bool)
    for p in range(seq[7]):
        at = int(c.table[7, p // page]), p % page
        k[at], mine[at] = math.nan, True
    got = dsa.key_weights(c.cfg, c.q.to(DEV), lse, k.to(DEV), c.table.to(DEV), i32(seq),
                          i32(c.cu), w, decay=0.5, w_out=torch.full_like(w, 7.0)).cpu()
    assert torch.equal(got[~mine], clean[~mine]) and got[mine].isnan().all()


@gpu
def test_weights_latch_bad_lengths_and_pages():
    c = Case([1, 1], [30, 30], 0, 8, 128, 16, 1, seed=51)
    for table, seq, cu in ((None, [30, 999], c.cu), (None, [-1, 30], c.cu), (None, c.seq, [0, 2, 1]),
                           (None, c.seq, [0, 1, 9]), (9999, c.seq, c.cu), (-3, c.seq, c.cu)):
        t = c.table.clone()
        if table is not None:
            t[0, 0] = table
        ws = dsa.serve_workspace(c.cfg, dsa.SERVE_WS_WEIGHTS, DEV)
        w = torch.zeros(c.k.shape[:2], device=DEV)
        k = torch.nan_to_num(c.k)
        dsa.key_weights(c.cfg, c.q.to(DEV), torch.zeros(2, 8, device=DEV), k.to(DEV), t.to(DEV),
                        i32(seq), i32(cu), w, ws=ws)
        assert dsa.get_device_status(ws) == 7, (table, seq, cu)
