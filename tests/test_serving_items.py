"""The shared-prefix attention where a pair of SMs has many tiles of a unit, or
many units: what a single-tile item never meets (the rescaling of O and of the
row sums, the P buffer's reuse, O's sum over tiles, the hand-over from item to
item), at every head dim, against the definition in fp64."""
import dataclasses
import math

import numpy as np
import pytest
import torch

from tests.test_serving import BF, Case
from tests.test_serving_scores import check_rows, plain_on_gpu, rows_of

gpu = pytest.mark.gpu


def spiked(c, kinds):
    """Exact integer scores at scale 1.  Row (t, h) looks at channels c and
    64 + c of the keys, c its number modulo 64.  Channel c is 15 at the keys j
    with j % 1024 == 16 c (spike A) and channel 64 + c is 30 at those with
    j % 1024 == (16 c + 520) % 1024 (spike B), else 0: e^15 is more than the 2^20
    past which a reference is raised, so a row meets A, and B behind it, once in
    every four tiles.  V of ordinary keys is 2^12 as large, and V of B's keys 2^-18,
    so that what came before a spike, A and B have like shares of O.  kinds[row in
    its block of 128] is 0: all scores alike, 1: spike A, 2: A and B."""
    d = c.q.shape[2]
    g = torch.Generator().manual_seed(7)
    c.cfg = dataclasses.replace(c.cfg, sm_scale=1.0)
    c.q[:] = 0
    q = c.q.view(-1, d)
    row = torch.arange(q.shape[0])
    kind = torch.tensor(kinds)[row % 128]
    for need, first in ((1, 0), (2, 64)):
        has = row[kind >= need]
        q[has, first + has % 64] = 1.0
    for b, n in [(-1, c.prefix)] + list(enumerate(c.seq)):
        at, j = rows_of(c, c.k, b, n), torch.arange(n)
        k = torch.zeros(n, d)
        a, z = j % 16 == 0, j % 16 == 8
        k[j[a], j[a] % 1024 // 16] = 15.0
        k[j[z], 64 + (j[z] - 520) % 1024 // 16] = 30.0
        size = torch.where(a, 1.0, torch.where(z, 2.0 ** -18, 2.0 ** 12))
        c.k.view(-1, d)[at] = k.to(BF)
        v = (1 + 0.25 * torch.randn((n, d), generator=g)) * size[:, None]
        c.v.view(-1, d)[at] = v.to(BF)
    return c


def check_twice(c):
    got = c.run()
    assert got[2] == 0
    check_rows(got, plain_on_gpu(c))
    again = c.run()
    n = c.cu[-1]
    assert torch.equal(got[0][:n], again[0][:n]) and torch.equal(got[1][:n], again[1][:n])


KINDS = {"all": [1 + r % 2 for r in range(128)],
         "low": [r % 3 if r < 64 else 0 for r in range(128)],
         "high": [r % 3 if r >= 64 else 0 for r in range(128)],
         "few": [2 if r in (3, 77) else 0 for r in range(128)]}


@gpu
@pytest.mark.parametrize("kinds", KINDS)
@pytest.mark.parametrize("d", [128, 256, 512])
def test_references_raised_inside_items(d, kinds):
    """Two and a half row blocks behind 60,000 keys, nine tiles a pair: spikes in
    every item's later tiles, in the last partial one, in one or both groups of 64
    rows, and a second, higher one behind the first."""
    check_twice(spiked(Case([1, 3, 1, 1], [2, 700, 33, 1], 60000, 50, d, 64, 2, seed=d),
                       KINDS[kinds]))


@gpu
@pytest.mark.parametrize("d", [128, 256, 512])
def test_references_raised_in_causal_items(d):
    """The same over the requests' own tokens: the last tiles are masked row by
    row."""
    check_twice(spiked(Case([2, 5, 1], [20001, 30000, 777], 0, 64, d, 32, 2, seed=d),
                       KINDS["all"]))


@gpu
@pytest.mark.parametrize("kv", [1, 2])
@pytest.mark.parametrize("d,B,H", [(128, 44, 128), (256, 21, 128), (512, 22, 64)])
def test_many_tiles_a_pair(d, B, H, kv):
    """More than 30 tiles a pair, in shares that begin and end inside units, and
    more rows than the joining kernel takes with several warps each."""
    r = np.random.default_rng(d)
    check_twice(Case([1] * B, r.integers(1, 900, B).tolist(), 60011, H, d, 64, kv, seed=d + kv))


@gpu
@pytest.mark.parametrize("kv", [1, 2])
@pytest.mark.parametrize("d", [128, 256, 512])
def test_many_items_a_pair(d, kv):
    """Four requests of a few rows for every pair, their own tokens up to three
    tiles, behind no prefix and behind one of two tiles."""
    r = np.random.default_rng(d)
    for prefix in (0, 400):
        new = r.integers(0, 3, 320).tolist()
        seq = [n + int(x) for n, x in zip(new, r.integers(0, 700, 320))]
        check_twice(Case(new, seq, prefix, 16, d, 32, kv, pad=3, seed=d + kv))


@gpu
@pytest.mark.parametrize("d", [256, 512])
def test_prompts_behind_a_prefix_and_alone(d):
    """Ragged prompts with their causal blocks, several items a pair."""
    check_twice(Case([700, 1, 350], [700, 90, 1200], 5003, 16, d, 64, 2, seed=d))
    check_twice(Case([1100, 333], [1100, 400], 0, 16, d, 128, 1, seed=d))
