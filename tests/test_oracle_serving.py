"""Pins of the serving oracle: hand-derived slots, adapters against a dense
weight, sampling against chances counted by hand and against enumeration."""

import math

import numpy as np
import pytest

from oracle import serving as O


def test_slots_by_hand():
    # page 16; a: 15 tokens + 2 (one new page), b: nothing new, c: empty + 17 (two pages), d: 16 + 16 (one)
    table = np.array([[5, 0], [6, 0], [0, 0], [7, 0]], np.int32)
    got = O.kv_slots(16, 100, table, [15, 3, 0, 16], [2, 0, 17, 16], [90, 91, 92, 93, 94], 1, 36)
    slots, pos, seq, lens, last, used, after = got
    assert after.tolist() == [[5, 91], [6, 0], [92, 93], [7, 94]]
    assert slots.tolist() == [95, 91 * 16] + [92 * 16 + i for i in range(16)] + [93 * 16] + [94 * 16 + i for i in range(16)] + [-1]
    assert pos.tolist() == [15, 16] + list(range(17)) + list(range(16, 32)) + [-1]
    assert seq.tolist() == [0] * 2 + [2] * 17 + [3] * 16 + [-1]
    assert lens.tolist() == [17, 3, 17, 32] and last.tolist() == [1, -1, 18, 34] and used.tolist() == [5]


def test_slots_refuse_what_does_not_fit():
    table = np.zeros((4, 2), np.int32)
    # two pages left: a takes one, b would need two more, c needs none, d again one
    got = O.kv_slots(16, 8, table, [0, 0, 3, 0], [16, 32, 1, 1], [3, 4], 0, 60)
    assert got[3].tolist() == [16, 0, 4, 0] and got[4].tolist() == [15, -1, 48, -1] and got[5].tolist() == [1]
    assert (got[0][16:48] == -1).all() and got[0][48] == 3
    # too long for the table, and past the step's rows, need no pages
    got = O.kv_slots(16, 8, table, [0, 30, 0, 0], [33, 2, 1, 9], [3, 4], 0, 36)
    assert got[3].tolist() == [0, 32, 1, 0] and got[5].tolist() == [1] and got[6][2, 0] == 3


def test_lora_is_a_dense_weight():
    rng = np.random.default_rng(1)
    a, b = rng.standard_normal((3, 8, 128)), rng.standard_normal((3, 5, 8))
    x, base, s = rng.standard_normal((4, 128)), rng.standard_normal((4, 5)), np.array([2.0, 0.5, -1.0])
    y, off = O.lora(a, b, x, [1, -1, 2, 3], base, s)
    assert np.allclose(y[0], base[0] + 0.5 * (b[1] @ a[1]) @ x[0]) and np.allclose(y[2], base[2] - (b[2] @ a[2]) @ x[2])
    assert (y[1] == base[1]).all() and (y[3] == base[3]).all() and (off[1] == 0).all() and (off[0] > 0).all()


def _chances(x, **kw):
    """How often each token comes up over evenly spaced u."""
    n = 4000
    ids = [O.sample(x, (i + 0.5) / n, **kw)[0] for i in range(n)]
    return np.bincount(ids, minlength=len(x)) / n


def test_sample_chances():
    x = np.log(np.array([1.0, 4.0, 2.0, 2.0, 1.0]))
    assert np.allclose(_chances(x), [.1, .4, .2, .2, .1], atol=1e-3)
    assert np.allclose(_chances(x, temperature=0.5), np.array([1, 16, 4, 4, 1]) / 26, atol=1e-3)
    assert np.allclose(_chances(x, top_k=2), np.array([0, 4, 2, 0, 0]) / 6, atol=1e-3)     # of equal ones the first
    assert np.allclose(_chances(x, top_p=0.4), [0, 1, 0, 0, 0], atol=1e-3)
    assert np.allclose(_chances(x, top_p=0.41), np.array([0, 4, 2, 0, 0]) / 6, atol=1e-3)
    assert np.allclose(_chances(x, top_p=0.0), [0, 1, 0, 0, 0], atol=1e-3)
    assert np.allclose(_chances(x, min_p=0.5), np.array([0, 4, 2, 2, 0]) / 8, atol=1e-3)
    # top-p over what top-k left: 4 / 6 is less than 0.7, so both stay
    assert np.allclose(_chances(x, top_k=2, top_p=0.7), np.array([0, 4, 2, 0, 0]) / 6, atol=1e-3)
    assert np.allclose(_chances(x, top_k=2, top_p=0.6), [0, 1, 0, 0, 0], atol=1e-3)


def test_sample_edges():
    inf, nan = math.inf, math.nan
    assert O.sample([3.0, 7.0, 7.0], 0.9, temperature=0.0) == (1, 0.0)
    assert O.sample([-inf, nan, -inf], 0.5) == (-1, -inf)
    assert O.sample([nan, 1.0, -inf], 0.99)[0] == 1
    assert O.sample([0.0, inf, 5.0, inf], 0.6) == (3, math.log(0.5))
    assert O.sample([0.0, 0.0], 1.0)[0] == 1 and O.sample([0.0, 0.0], nan)[0] == 0
    assert O.sample([0.0, -0.0, 0.0], 0.5, top_k=1)[0] == 0


@pytest.mark.parametrize("seed", range(4))
def test_sample_against_enumeration(seed):
    """Every token's share of u against its weight among the kept, found by
    comparing every pair of tokens instead of sorting."""
    rng = np.random.default_rng(seed)
    n = 12
    x = rng.integers(-3, 4, n).astype(np.float64)
    k, p, m, t = int(rng.integers(1, n)), float(rng.uniform(0.2, 0.95)), float(rng.uniform(0, 0.3)), 1.3
    ahead = np.array([[x[j] > x[i] or (x[j] == x[i] and j < i) for j in range(n)] for i in range(n)])
    w = np.exp((x - x.max()) / t)
    kept = ahead.sum(1) < k
    total = w[kept].sum()
    kept &= np.array([(ahead[i] * kept) @ w for i in range(n)]) < p * total
    kept &= w >= m
    want = np.where(kept, w, 0) / w[kept].sum()
    assert np.allclose(_chances(x, temperature=t, top_k=k, top_p=p, min_p=m), want, atol=1e-3)
    for u in (0.05, 0.5, 0.95):
        i, lp = O.sample(x, u, temperature=t, top_k=k, top_p=p, min_p=m)
        assert abs(lp - math.log(want[i])) < 1e-12


def test_slots_used_counts_pages_given_out():
    """One page left, asked for by a sequence that needs two, before one that needs none."""
    out = O.kv_slots(16, 8, np.array([[0, -1, -1], [1, -1, -1]], np.int32), np.array([16, 3], np.int32),
                     np.array([17, 1], np.int32), np.array([5], np.int32), 0, 18)
    assert out[5].tolist() == [0] and out[3].tolist() == [16, 4] and out[6].tolist() == [[0, -1, -1], [1, -1, -1]]
