"""Log probabilities of given tokens, entropy and alternatives, and their
gradient, against plain definitions in fp64."""
import ctypes
import math

import pytest
import torch

import long_context_sparse_gb300 as dsa
from long_context_sparse_gb300 import build as dsa_build
from tests.test_serving import DEV
from tests.test_tree import P, i32

gpu = pytest.mark.gpu
TYPES = [torch.bfloat16, torch.float16, torch.float32]


# ----------------------------------------------------- plain definitions


def plain(logits, tokens, n_top, scale):
    """fp64 (logp, lse, entropy, ids, top_logp)."""
    x = logits.double()
    ids = torch.sort(x + 0.0, dim=1, descending=True, stable=True)[1][:, :n_top]
    x = x * scale
    # from the row's maximum: at 1e38 even fp64 has no room for log V beside it
    m = x.amax(1, keepdim=True)
    none = m[:, 0] == -math.inf
    z = x - torch.where(m == -math.inf, 0.0, m)
    total = torch.exp(z).sum(1, keepdim=True).log()
    y, lse = z - total, (m + total)[:, 0]
    p = torch.exp(y)
    ent = -torch.where(p > 0, p * y, 0.0).sum(1)
    ent[none] = 0.0
    ent[torch.isnan(lse) | (lse == math.inf)] = math.nan
    y = torch.where(none[:, None], -math.inf, y)
    t = tokens.long()
    logp = torch.where(t >= 0, y.gather(1, t.clamp(min=0)[:, None])[:, 0], 0.0)
    return logp, lse, ent, ids, y.gather(1, ids)


def bounds(logits, lse, entropy, scale):
    """What fp32 may add, from the kernel's steps: y = (x - r) c with two roundings
    (2^-23 |y|) and 2^y with 2^-22 leave each term off by 2^-22 (1 + |y|), weighted by
    the terms themselves: sum p |y| ln 2 = lse - max - entropy at the row's maximum, and
    terms beyond 2^-126 of it are nothing; a thread adds V / 256 of them and the rest
    of the sum is a tree; the result is rounded once more."""
    V = logits.shape[1]
    top = logits.double().amax(1) * scale
    spread = (lse - top - entropy).abs() / math.log(2) + 1
    rel = 2.0 ** -22 * (1 + spread) + (V / 256 + 64) * 2.0 ** -24
    at = 2.0 ** -22 * (top.abs() + lse.abs())
    return rel + at, rel * (1 + 2 * spread) + 2.0 ** -22 * (1 + spread)


def check(logits, tokens, n_top, scale, out=None, ws=None):
    ws = dsa.logprobs_workspace(DEV) if ws is None else ws
    got = dsa.token_logprobs(logits, tokens, n_top, scale, out=out, ws=ws)
    assert dsa.get_device_status(ws) == 0
    rows = logits.shape[0]
    assert got.top_ids.shape == (rows, n_top) and got.top_logp.shape == (rows, n_top)
    c = logits.cpu()
    logp, lse, ent, ids, top = plain(c, tokens.cpu(), n_top, scale)
    fine = torch.isfinite(lse)
    l_tol, h_tol = bounds(c[fine], lse[fine], ent[fine], scale)
    g = [t.cpu().double() for t in (got.logp, got.lse, got.entropy, got.top_logp)]
    assert torch.equal(got.top_ids.cpu().long(), ids) or not fine.all()
    assert torch.equal(got.top_ids.cpu().long()[fine], ids[fine])

    def close(a, b, tol, name):
        same = (a == b) | ((a - b).abs() <= tol + 2.0 ** -22 * b.abs())
        assert same.all(), f"{name}: {(a - b).abs().max():.3g}"

    close(g[1][fine], lse[fine], l_tol, "lse")
    close(g[0][fine], logp[fine], l_tol, "logp")
    close(g[2][fine], ent[fine], h_tol, "entropy")
    close(g[3][fine], top[fine], l_tol[:, None], "top_logp")
    assert (g[2][fine] >= -1e-5).all()
    none = lse == -math.inf
    assert (g[1][none] == -math.inf).all() and (g[2][none] == 0).all()
    assert (g[3][none] == -math.inf).all()
    assert (g[0][none] == torch.where(tokens.cpu()[none] < 0, 0.0, -math.inf)).all()
    bad = ~fine & ~none
    assert torch.isnan(g[1][bad]).all() and torch.isnan(g[2][bad]).all()
    assert torch.isnan(g[3][bad]).all()
    i = got.top_ids.cpu()
    assert ((i >= 0) & (i < logits.shape[1])).all()
    return got


def logits_of(rows, vocab, dtype, seed, spread=3.0, ld=None, shift=0):
    g = torch.Generator().manual_seed(seed)
    full = (spread * torch.randn((rows, (ld or vocab) + shift), generator=g)).to(dtype)
    tok = torch.randint(0, vocab, (rows,), generator=g, dtype=torch.int32)
    return full.to(DEV)[:, shift:shift + vocab], tok.to(DEV)


# ------------------------------------------------------------ host checks


@pytest.fixture(scope="module")
def lib():
    dsa_build.build()
    return dsa._load()


def config(**kw):
    base = dict(rows=4, vocab=100, ld=104, dtype=0, n_top=2, scale=1.0, reserved=0)
    base.update(kw)
    return dsa._CLogprobsConfig(*base.values())


def test_layout():
    C = dsa._CLogprobsConfig
    assert ctypes.sizeof(C) == 40 and C.dtype.offset == 24 and C.scale.offset == 32


FWD = dict(logits=4 * 104 * 2, tokens=16, logp=16, lse=16, entropy=16, ids=32, top=32, ws=256)
BWD = dict(logits=4 * 104 * 2, tokens=16, lse=16, entropy=16, g=16, h=16, dx=4 * 104 * 2)


def fwd(lib, at, ws_bytes=256, cfg=None, **over):
    a = {**at, **over}
    cfg = config() if cfg is None else cfg
    return lib.dsa_token_logprobs(ctypes.byref(cfg), *(P(x) for x in a.values()), ws_bytes, None)


def bwd(lib, at, ld=104, ws=1 << 40, ws_bytes=256, cfg=None, **over):
    a = {**at, **over}
    cfg = config() if cfg is None else cfg
    return lib.dsa_token_logprobs_bwd(ctypes.byref(cfg), *(P(x) for x in a.values()), ld, P(ws),
                                      ws_bytes, None)


@pytest.mark.parametrize("over,code", [
    (dict(rows=0), 1), (dict(vocab=0), 1), (dict(ld=99), 1), (dict(dtype=3), 1),
    (dict(dtype=-1), 1), (dict(n_top=-1), 1), (dict(vocab=1, n_top=2), 1), (dict(scale=0.0), 1),
    (dict(scale=-1.0), 1), (dict(scale=math.inf), 1), (dict(scale=math.nan), 1),
    (dict(scale=2.4e38), 1), (dict(reserved=1), 1), (dict(n_top=65), 2), (dict(rows=1 << 31), 2),
    (dict(vocab=1 << 30, ld=1 << 30), 2), (dict(ld=1 << 40), 2)])
def test_configs_refused(lib, over, code):
    at = {n: (i + 1) << 28 for i, n in enumerate(FWD)}
    assert fwd(lib, at, cfg=config(**over)) == code
    at = {n: (i + 1) << 28 for i, n in enumerate(BWD)}
    assert bwd(lib, at, cfg=config(**over), ld=1 << 30) == code


def test_buffers_refused(lib):
    at = {n: (i + 1) << 28 for i, n in enumerate(FWD)}
    for w in ("logp", "lse", "entropy", "ids", "top", "ws"):
        for x in FWD:
            if x != w:
                assert fwd(lib, at, **{w: at[x]}) == 1, (w, x)
    for x in FWD:
        assert fwd(lib, at, **{x: None}) == 1, x
        if x not in ("logits", "ws"):
            assert fwd(lib, at, **{x: at[x] + 2}) == 4, x
    none = config(n_top=0)
    assert fwd(lib, at, cfg=none) == 1                     # alternatives, but none wanted
    assert fwd(lib, at, logits=at["logits"] + 1) == 4
    assert fwd(lib, at, logits=at["logits"] + 2, cfg=config(dtype=2)) == 4
    assert fwd(lib, at, ws_bytes=255) == 3 and fwd(lib, at, ws=at["ws"] + 16) == 4
    at = {n: (i + 1) << 28 for i, n in enumerate(BWD)}
    for x in BWD:
        if x != "dx":
            assert bwd(lib, at, dx=at[x] + (16 if x == "logits" else 0)) == 1, x
            assert bwd(lib, at, ws=at[x]) == 1, x
        if x not in ("entropy", "g", "h"):
            assert bwd(lib, at, **{x: None}) == 1, x
    assert bwd(lib, at, entropy=None) == 1                 # its gradient needs it
    assert bwd(lib, at, ld=99) == 1 and bwd(lib, at, ld=1 << 40) == 2
    assert bwd(lib, at, dx=at["logits"], ld=112) == 1      # in place, another stride
    assert bwd(lib, at, dx=at["dx"] + 1) == 4 and bwd(lib, at, g=at["g"] + 2) == 4
    assert bwd(lib, at, ws_bytes=255) == 3


def test_python_refuses_wrong_logits():
    t = torch.zeros(3, dtype=torch.int32)
    with pytest.raises(ValueError):
        dsa.token_logprobs(torch.zeros(3, 5), t)


# --------------------------------------------------------------- forward


@gpu
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("vocab", [1, 2, 7, 8, 9, 16, 31, 257, 2048, 4099, 50257, 131072, 200001])
def test_logprobs(dtype, vocab):
    for rows, n_top, pad, shift in ((3, min(vocab, 5), 0, 0), (1, min(vocab, 64), 3, 1),
                                    (700 if vocab < 5000 else 5, min(vocab, 20), 1, 3)):
        x, tok = logits_of(rows, vocab, dtype, vocab + rows, ld=vocab + pad, shift=shift)
        check(x, tok, n_top, 0.7 if rows == 3 else 1.0)


@gpu
def test_rows_that_fill_the_gpu():
    """A CTA a row, and clusters of two, four and eight: the same results."""
    x, tok = logits_of(1300, 40000, torch.bfloat16, 1)
    for rows in (1300, 650, 310, 160, 80, 3):
        check(x[:rows], tok[:rows], 20, 1.0)
    check(x[:200], tok[:200], 0, 1.0)


@gpu
@pytest.mark.parametrize("dtype", TYPES)
def test_masked_and_special_rows(dtype):
    V = 5000
    x, tok = logits_of(40, V, dtype, 3)
    x[0, ::2] = -math.inf
    x[1, 5:] = -math.inf                      # fewer finite ones than alternatives
    x[2] = -math.inf
    x[3] = torch.finfo(dtype).min
    x[4, :] = torch.finfo(dtype).min
    x[4, 77] = 0.0
    x[5, 9] = math.nan
    x[6, 9] = math.inf
    x[7] = math.nan
    x[8, :4990] = -math.inf                   # the tail alone
    x[9, 1:] = -math.inf                      # the first alone
    x[10] = 0.0
    x[10, ::3] = -0.0                         # alike
    x[11] = 1.5                               # all equal
    x[12] = torch.finfo(dtype).max / 8
    tok[13], tok[2], tok[14] = -1, -7, 4999
    tok[0] = 0                                # a masked token
    check(x, tok, 10, 1.0)
    check(x, tok, 64, 0.25)
    check(x[2:3], tok[2:3], 64, 1.0)
    check(x[11:12], tok[11:12], 64, 1.0)


@gpu
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("vocab", [3000, 70000, 131072])
def test_alternatives_in_awkward_places(dtype, vocab):
    """Many of the best in one thread's elements, ascending and descending rows, few
    different values."""
    rows = 8
    x, tok = logits_of(rows, vocab, dtype, vocab, spread=1.0)
    per = 16 // x.element_size()
    lanes = torch.arange(0, vocab, 256 * per, device=DEV)          # thread 0's vectors
    x[0, lanes] = 20.0 + torch.arange(len(lanes), device=DEV).to(dtype) * 0.125
    for e in range(per):
        x[1, (lanes + e).clamp(max=vocab - 1)] = 30.0              # and all of them alike
    x[2] = torch.linspace(-8, 8, vocab, device=DEV).to(dtype)
    x[3] = torch.linspace(8, -8, vocab, device=DEV).to(dtype)
    x[4] = torch.randint(0, 3, (vocab,), device=DEV).to(dtype)
    x[5] = 0.0
    x[5, -30:] = 5.0
    x[6] = torch.arange(vocab, device=DEV).remainder(17).to(dtype)
    x[7, : vocab // 2] = 7.0
    for n_top in (1, 20, 64):
        check(x, tok, n_top, 1.0)
    many = x.repeat(100, 1)[:, : min(vocab, 40000)]
    check(many, tok.repeat(100).clamp(max=many.shape[1] - 1), 33, 1.0)


@gpu
def test_large_logits_and_scales():
    for dtype, size in ((torch.float32, 1e30), (torch.bfloat16, 1e30), (torch.float16, 6e4)):
        x, tok = logits_of(6, 3001, dtype, 5, spread=1.0)
        x = (x.float() * size / 5).to(dtype)
        check(x, tok, 4, 1.0)
        check(x, tok, 4, 1e-6)
    x, tok = logits_of(6, 3001, torch.float32, 6)
    check(x, tok, 4, 1e4)
    check(x + 1000.0, tok, 4, 1.0)


@gpu
def test_tokens_out_of_range_are_latched():
    x, tok = logits_of(5, 100, torch.float32, 7)
    tok[3] = 100
    ws = dsa.logprobs_workspace(DEV)
    got = dsa.token_logprobs(x, tok, ws=ws)
    assert dsa.get_device_status(ws) == 7 and got.logp[3] == 0 and (got.logp[:3] < 0).all()
    z = torch.zeros(5, device=DEV)
    d = dsa.token_logprobs_bwd(x, tok, got.lse, got.entropy, z + 1, ws=ws)
    assert dsa.get_device_status(ws) == 7
    assert (d[3] == 0).all() and (d[2] != 0).any()


# -------------------------------------------------------------- gradient


def plain_grad(x, tok, lse, ent, g, h, scale):
    """fp64 gradient, and the sum of the sizes of its terms."""
    y = x.double() * scale - lse.double()[:, None]
    p = torch.exp(y)
    y = torch.where(p > 0, y, 0.0)
    one = torch.zeros_like(y)
    live = tok >= 0
    one[live, tok[live].long()] = 1.0
    g = torch.where(live, g.double(), 0.0)[:, None]
    h, e = h.double()[:, None], ent.double()[:, None]
    d = scale * (g * (one - p) - h * p * (y + e))
    size = scale * (g.abs() * (one + p) + h.abs() * p * (y.abs() + e.abs()))
    none = (lse == -math.inf)[:, None]
    return torch.where(none, 0.0, d), torch.where(none, 0.0, size), y


def check_grad(x, tok, scale, seed, dx=None, use=(True, True)):
    g = torch.Generator().manual_seed(seed)
    rows = x.shape[0]
    up = [torch.randn(rows, generator=g) if u else torch.zeros(rows) for u in use]
    _, lse, ent, _, _ = plain(x.cpu(), tok.cpu(), 0, scale)
    lse, ent = lse.float(), ent.float()
    d, size, y = plain_grad(x.cpu(), tok.cpu(), lse, ent, *up, scale)
    ws = dsa.logprobs_workspace(DEV)
    dev = lambda t: t.to(DEV)
    got = dsa.token_logprobs_bwd(x, tok, dev(lse), dev(ent) if use[1] else None,
                                 dev(up[0]) if use[0] else None, dev(up[1]) if use[1] else None,
                                 scale, dlogits=dx, ws=ws)
    assert dsa.get_device_status(ws) == 0 and got.dtype == x.dtype
    # half a step of the type; fp32: log p off by 2^-24 (|log p| + |scale x|), its
    # product with log2(e), 2^ and the factors by 2^-22 and 2^-23 (1 + |log p|)
    lim = torch.finfo(x.dtype)
    rel = 2.0 ** -20 + 2.0 ** -22 * y.abs() + 2.0 ** -24 * torch.nan_to_num(
        (x.cpu().double() * scale).abs(), posinf=0.0)
    err = (got.cpu().double() - d).abs()
    assert (err <= lim.eps / 2 * d.abs() + size * rel + lim.tiny * lim.eps).all(), \
        f"{(err / (d.abs() + 1e-30)).max():.3g}"
    return got


@gpu
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("vocab", [1, 2, 7, 8, 9, 257, 8192, 8193, 50257])
def test_gradient(dtype, vocab):
    for rows, pad, shift, scale in ((3, 0, 0, 1.0), (9, 3, 1, 0.6), (2, 8, 8, 1.0)):
        x, tok = logits_of(rows, vocab, dtype, vocab + rows, ld=vocab + pad, shift=shift)
        check_grad(x, tok, scale, rows)
        odd = torch.full((rows, vocab + 7), 9.0, dtype=dtype, device=DEV)
        got = check_grad(x, tok, scale, rows, dx=odd[:, 3:3 + vocab])   # another place in 16 bytes
        assert got.data_ptr() == odd[:, 3:].data_ptr()
        assert (odd[:, :3] == 9).all() and (odd[:, 3 + vocab:] == 9).all()


@gpu
@pytest.mark.parametrize("use", [(True, False), (False, True), (False, False)])
def test_gradient_of_one_output(use):
    x, tok = logits_of(5, 1000, torch.float32, 8)
    got = check_grad(x, tok, 1.0, 3, use=use)
    assert use[0] or use[1] or (got == 0).all()


@gpu
@pytest.mark.parametrize("dtype", TYPES)
def test_gradient_in_place_masked_and_without_tokens(dtype):
    x, tok = logits_of(12, 3001, dtype, 9)
    x[0, ::2] = -math.inf
    x[1] = -math.inf
    x[2, 1:] = -math.inf
    tok[3], tok[0], tok[2] = -1, 1, 0
    got = check_grad(x, tok, 1.0, 4)
    assert (got[1] == 0).all() and (got[0, ::2] == 0).all()
    y = x.clone()
    again = check_grad(y, tok, 1.0, 4, dx=None)
    lse = torch.logsumexp(x.double(), 1).float()
    ent = plain(x.cpu(), tok.cpu(), 0, 1.0)[2].float().to(DEV)
    g = torch.ones(12, device=DEV)
    want = dsa.token_logprobs_bwd(x, tok, lse, ent, g, g)
    assert dsa.token_logprobs_bwd(y, tok, lse, ent, g, g, dlogits=y) is y
    assert torch.equal(y, want) and torch.equal(again, got)


@gpu
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("shift", [0, 1])
def test_rows_without_gradient_are_zero_whatever_their_logits(dtype, shift):
    """Padding rows: logits, lse and entropy that are not numbers, no token or a
    gradient of 0, on both ways to read the logits."""
    x, tok = logits_of(8, 1003, dtype, 12)
    x[1], x[2, 5], x[3] = math.nan, math.inf, torch.finfo(dtype).max
    tok[1], tok[3] = -1, -1
    g, h = torch.ones(8, device=DEV), torch.ones(8, device=DEV)
    h[1:4], g[2] = 0.0, 0.0
    p = dsa.token_logprobs(x, tok)
    out = torch.full((8, 1003 + shift), 9.0, dtype=dtype, device=DEV)[:, shift:]
    dsa.token_logprobs_bwd(x, tok, p.lse, p.entropy, g, h, dlogits=out)
    assert (out[1:4] == 0).all() and out[[0, 4, 5, 6, 7]].isfinite().all()
    assert (out[[0, 4, 5, 6, 7]] != 0).any(1).all()
    dsa.token_logprobs_bwd(x, tok, p.lse, None, g, dlogits=out)
    assert (out[1:4] == 0).all()
    y = x.clone()
    dsa.token_logprobs_bwd(y, tok, p.lse, p.entropy, g, h, dlogits=y)
    assert (y[1:4] == 0).all()


@gpu
def test_gradient_against_differences_and_the_forward():
    """The kernels' own lse and entropy into the kernel's gradient; against central
    differences in fp64 and against autograd through the definition."""
    x, tok = logits_of(4, 23, torch.float32, 10, spread=1.5)
    scale, rows = 0.8, 4
    f = dsa.token_logprobs(x, tok, scale=scale)
    g = torch.tensor([1.0, -0.5, 2.0, 0.0])
    h = torch.tensor([0.3, 1.0, 0.0, -2.0])
    d = dsa.token_logprobs_bwd(x, tok, f.lse, f.entropy, g.to(DEV), h.to(DEV), scale).cpu().double()

    def loss(z):
        y = torch.log_softmax(z * scale, 1)
        ent = -(y.exp() * y).sum(1)
        return (g * y[torch.arange(rows), tok.cpu().long()] + h * ent).sum()

    z = x.cpu().double().requires_grad_()
    loss(z).backward()
    assert (d - z.grad).abs().max() <= 2e-6      # 2^-20 of terms below 2
    with torch.no_grad():
        for r in range(rows):
            for j in range(23):
                e = torch.zeros_like(z)
                e[r, j] = 1e-4
                diff = (loss(z + e) - loss(z - e)) / 2e-4
                assert abs(diff - d[r, j]) <= 3e-6   # 1e-8 of curvature on top


# ------------------------------------------------------------- in place


@gpu
def test_offsets_past_32_bits():
    """The last rows of a tensor of more than 2^31 elements, and of a long stride."""
    V = 131072
    rows = (1 << 31) // V + 5
    x = torch.zeros((rows, V), dtype=torch.bfloat16, device=DEV)
    y, tok = logits_of(5, V, torch.bfloat16, 11)
    x[-5:] = y
    full = torch.zeros(rows, dtype=torch.int32, device=DEV)
    full[-5:] = tok
    got = dsa.token_logprobs(x, full, n_top=5)
    want = check(y, tok, 5, 1.0)
    for a, b in zip(got, want):
        assert (a[-5:].double() - b.double()).abs().max() <= 1e-4
    assert torch.equal(got.top_ids[-5:], want.top_ids)
    g = torch.ones(rows, device=DEV)
    d = dsa.token_logprobs_bwd(x, full, got.lse, got.entropy, g, dlogits=x)
    e = dsa.token_logprobs_bwd(y, tok, got.lse[-5:].clone(), got.entropy[-5:].clone(), g[:5])
    assert torch.equal(d[-5:], e)


@gpu
def test_streams_devices_and_graphs():
    x, tok = logits_of(64, 30000, torch.bfloat16, 12)
    ref = dsa.token_logprobs(x, tok, n_top=8)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    ws, out = dsa.logprobs_workspace(DEV), [torch.empty_like(t) for t in ref]
    out = dsa.TokenLogprobs(*out)
    with torch.cuda.stream(s):
        dsa.token_logprobs(x, tok, n_top=8, out=out, ws=ws)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(out, ref))
    one = torch.ones(64, device=DEV)
    dx = torch.empty_like(x)
    step = lambda: (dsa.token_logprobs(x, tok, n_top=8, out=out, ws=ws),
                    dsa.token_logprobs_bwd(x, tok, out.lse, out.entropy, one, one, dlogits=dx,
                                           ws=ws))
    step()
    torch.cuda.synchronize()
    want = dx.clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for _ in range(3):
        dx.zero_()
        for t in out:
            t.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(dx, want) and all(torch.equal(a, b) for a, b in zip(out, ref))
