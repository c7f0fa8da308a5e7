"""The shared-prefix attention where scores are large, infinite or not numbers,
against the definition in fp64."""
import dataclasses
import math

import pytest
import torch

from tests.test_serving import LSE_TOL, O_TOL, P_TOL, BF, DEV, Case

gpu = pytest.mark.gpu


def rows_of(c, x, b, n):
    """Positions in x.view(-1, d) of the first n tokens of request b, or of the
    prefix (b = -1)."""
    page = c.cfg.page_size
    pages = (c.prefix_table if b < 0 else c.table[b]).long()
    j = torch.arange(n)
    return pages[j // page] * page + j % page


def plain_on_gpu(c):
    """As plain_attn, on the GPU a request at a time: (O, LSE, sum_j P_j |v_j|) in
    fp64, NaN for rows of no request."""
    T, H, d = c.q.shape
    o = torch.full((T, H, d), math.nan, dtype=torch.float64, device=DEV)
    mag, lse = o.clone(), torch.full((T, H), math.nan, dtype=torch.float64, device=DEV)

    def take(x, b, n):
        return x.reshape(-1, d)[rows_of(c, x, b, n)].to(DEV).double()

    kp, vp = take(c.k, -1, c.prefix), take(c.v, -1, c.prefix)
    for b, n in enumerate(c.seq):
        new, at = c.cu[b + 1] - c.cu[b], c.cu[b]
        if new == 0:
            continue
        q = c.q[at:at + new].to(DEV).double()
        last = (n - new + torch.arange(new, device=DEV)).clamp(min=-1)
        unseen = torch.arange(n, device=DEV)[None, :] > last[:, None]
        own = (q @ take(c.k, b, n).T).masked_fill(unseen[:, None, :], -math.inf)
        s = torch.cat([q @ kp.T, own], -1) * c.cfg.scale
        p = torch.softmax(s, -1)
        p = torch.where((s == -math.inf).all(-1, keepdim=True), 0.0, p)
        vo = take(c.v, b, n)
        for out, w in ((o, lambda x: x), (mag, torch.abs)):
            out[at:at + new] = p[..., :c.prefix] @ w(vp) + p[..., c.prefix:] @ w(vo)
        lse[at:at + new] = torch.logsumexp(s, -1)
    return o.cpu(), lse.cpu(), mag.cpu()


def check_rows(got, ref):
    """Every row of a request by its own size: O as in test_serving, LSE within
    what the scores' error makes of it and fp32's share of its own size."""
    o, lse = got[0].double(), got[1].double()
    ro, rl, mag = ref
    live = ~torch.isnan(rl[:, 0])
    o, lse, ro, rl, mag = (x[live] for x in (o, lse, ro, rl, mag))
    empty = rl == -math.inf
    assert torch.equal(lse[empty], rl[empty]) and (o[empty] == 0).all()
    o, lse, ro, rl, mag = (x[~empty] for x in (o, lse, ro, rl, mag))
    assert torch.isfinite(o).all() and torch.isfinite(lse).all()
    err = (o - ro).abs() - O_TOL * ro.abs() - P_TOL * mag
    assert (err <= 1e-30).all(), f"O: {err.max():.3g} over the bound"
    err = (lse - rl).abs() - LSE_TOL - 2.0 ** -22 * rl.abs()
    assert (err <= 0).all(), f"LSE: {err.max():.3g} over the bound"


def scored(c, rows, scale, fill):
    """c with scores that are exact in fp32: q is rows[h % len(rows)] in dim 0 and
    0 elsewhere, and dim 0 of the keys is fill(request or -1, number of keys)."""
    c.cfg = dataclasses.replace(c.cfg, sm_scale=scale)
    c.q[:] = 0
    for h in range(c.q.shape[1]):
        c.q[:, h, 0] = rows[h % len(rows)]
    flat = c.k.view(-1, c.k.shape[-1])
    for b, n in [(-1, c.prefix)] + list(enumerate(c.seq)):
        flat[rows_of(c, c.k, b, n), 0] = fill(b, n).to(BF)
    return c


@gpu
@pytest.mark.parametrize("scale", [1.0, 0.0])
@pytest.mark.parametrize("n_low", [33, 300, 1999])
@pytest.mark.parametrize("low,best", [(-1e9, 20), (-1e9, 30), (-1e9, 100), (-1e12, 5),
                                      (-1e12, 100), (-3e38, 5), (-3e38, 100)])
def test_first_keys_far_below_the_rest(low, best, n_low, scale):
    """The first keys of each list lie at a mask's value, written into a channel
    of the key, and the best scores are 5 to 100.  For some rows the mask's keys
    are the best by far instead, or count like all others."""
    g = torch.Generator().manual_seed(n_low)

    def fill(b, n):
        x = torch.tensor([0.25 * best, best - 3.0, best])[torch.randint(3, (n,), generator=g)]
        x[:n_low if b < 0 else min(n_low, n // 2)] = low
        return x

    c = scored(Case([1, 2], [40, 700], 2000, 16, 512, 64, 2, seed=n_low),
               [1.0, 0.5, 0.0, -1.0], scale, fill)
    got = c.run()
    assert got[2] == 0
    check_rows(got, plain_on_gpu(c))


@gpu
@pytest.mark.parametrize("d", [128, 512])
@pytest.mark.parametrize("n_low", [1, 32, 33, 300, 2000])
@pytest.mark.parametrize("rest", [-1000.0, -200.0, 0.0, 100.0])
def test_first_keys_at_minus_infinity(rest, n_low, d):
    """The first keys of the prefix score -inf and the rest far below or above 0.
    Request 0 of three has nothing else, where the whole prefix scores -inf."""
    def fill(b, n):
        x = torch.full((n,), rest)
        x[:n_low if b < 0 else (n if b == 0 else n // 2)] = -math.inf
        return x

    c = scored(Case([1, 2, 1], [40, 700, 3], 2000, 16, d, 64, 2, seed=n_low),
               [1.0, 0.5, 2.0], 1.0, fill)
    got = c.run()
    assert got[2] == 0
    check_rows(got, plain_on_gpu(c))


@gpu
@pytest.mark.parametrize("prefix", [0, 100, 300, 2000])
@pytest.mark.parametrize("value", [math.nan, math.inf])
def test_rows_that_are_not_numbers_stay_so(value, prefix):
    """A query row of NaN (or with an infinite channel, which makes scores of both
    signs infinite) is NaN in O and LSE, whatever tiles it meets; the rows beside
    it are as they would be without."""
    c = Case([2, 1], [300, 40], prefix, 16, 512, 64, 1, seed=prefix)
    ref = c.plain()
    bad = [(0, 0), (0, 15), (1, 3), (2, 7)]
    for t, h in bad:
        if math.isnan(value):
            c.q[t, h] = value
        else:
            c.q[t, h, 5] = value
    o, lse, st = c.run()
    assert st == 0
    for t, h in bad:
        assert torch.isnan(o[t, h]).all() and torch.isnan(lse[t, h]), (t, h)
        o[t, h], lse[t, h] = ref[0][t, h].to(BF), ref[1][t, h].float()
    check_rows((o, lse), ref)


@gpu
@pytest.mark.parametrize("kv", [1, 2])
@pytest.mark.parametrize("value", [math.nan, math.inf])
def test_a_token_that_is_not_finite_stays_in_its_request(value, kv):
    """The last own token of the middle request is not finite: its own rows may
    be anything, the other requests' are as they would be without."""
    c = Case([2, 3, 2], [300, 40, 70], 500, 16, 256, 32, kv, seed=kv)
    ref = c.plain()
    at = rows_of(c, c.v, 1, 40)[-1]
    c.v.view(-1, 256)[at, ::3] = value
    o, lse, st = c.run()
    assert st == 0
    others = [0, 1, 5, 6]
    check_rows((o[others], lse[others]), [x[others] for x in ref])
