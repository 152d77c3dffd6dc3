"""wq_sample where parts of a row lie far below its largest logit, or far from
zero: what is drawn is a token of the row that is kept, close to where the
draw falls, and its log chance within the bound of the sums."""

import math

import numpy as np
import pytest
import torch

import dequant_gemv_rht_amd as dq
from oracle import serving as O

from gpu_util import dev, say

pytestmark = pytest.mark.gpu


def check_near(x, u, unit=44, **kw):
    """Every row's token and log chance against what is kept in 64 bits; weights are counted in 2^-unit."""
    rows = len(x)
    ids, logp = dq.wq_sample(dev(x), dev(u), **{n: dev(np.full(rows, v, np.int32 if n == "top_k" else np.float32))
                                                for n, v in kw.items()})
    kw = {n: v if n == "top_k" else float(np.float32(v)) for n, v in kw.items()}
    same = (x == x[0]).all()   # rows that only their draws tell apart
    for r, (i, lp) in enumerate(zip(ids.tolist(), logp.tolist())):
        if r == 0 or not same:
            place, w = O.kept(x[r], **kw)
            up_to, total = np.cumsum(w), w.sum()
        at = np.flatnonzero(place == i)
        assert len(at) == 1, f"row {r}: token {i} is not kept ({kw})"
        # A weight is off by 2^-34 of itself and half of a unit at most (the
        # largest is one or more of 2^unit), so a sum of the n kept by 2^-34 of
        # itself and n 2^-45 (unit 44), and the draw, u of all of them, by as much; the log of a share by both
        # sums' relative errors (all is at least 1), then a 32-bit rounding.
        off = 2 * (2.0 ** -34 * total + len(w) * 2.0 ** -(unit + 1))
        draw = (min(max(float(u[r]), 0.0), 1.0) if u[r] == u[r] else 0.0) * total
        mine, after = w[at[0]], float(up_to[at[0]])
        assert after - mine - off <= draw <= after + off, f"row {r}: {i}, {after - draw} from the draw ({kw})"
        want = math.log1p(-(total - mine) / total) if mine > total - mine else math.log(mine / total)
        assert abs(lp - want) <= 2 * (2.0 ** -34 + len(w) * 2.0 ** -(unit + 1)) + abs(want) * (2.0 ** -33 + 2.0 ** -24), \
            f"row {r}: {lp} for {want} ({kw})"
    return ids.tolist()


DRAWS = np.array([0.0, math.nan, -1.0, 2.0 ** -33, 2.0 ** -24, 0.5, 1 - 2.0 ** -24, 1.0, 7.0], np.float32)


@pytest.mark.parametrize("half", [False, True])
@pytest.mark.parametrize("vocab", [16384, 20000, 40001])
@pytest.mark.parametrize("powers", [40.0, 44.0, 45.0, 45.3, 46.0, 46.6, 50.0, 54.0, 56.0, 58.0, 63.0, 70.0])
def test_whole_parts_far_below_the_largest(powers, vocab, half):
    """One large weight in one part, thousands of equal small ones before or behind it, draws at both ends."""
    rows, t = len(DRAWS), np.float16 if half else np.float32
    low = t(3.0 - math.log(2.0) * powers)
    for place in (vocab - 1, 8192 + 100, 100):
        x = np.full((rows, vocab), low, t)
        x[:, place] = 3.0
        say("sample", powers, vocab, half, place)
        ids = check_near(x, DRAWS)
        if powers <= 54:   # 8192 of 2^-54 are 8 units: the ends of the row are drawn
            if place >= 8192:
                assert ids[:3] == [0, 0, 0]
            if place < 8192:
                assert ids[-2:] == [vocab - 1] * 2
        for kw in (dict(temperature=1.0), dict(top_k=1), dict(top_k=5), dict(top_k=9000), dict(top_k=vocab - 1),
                   dict(top_p=1 - 2.0 ** -24), dict(top_p=0.5), dict(min_p=1e-30), dict(min_p=0.5),
                   dict(top_k=9000, top_p=1 - 2.0 ** -24, min_p=1e-14)):
            check_near(x, DRAWS, **kw)


@pytest.mark.parametrize("powers", [(20.0, 60.0), (43.0, 49.0), (46.0, 57.0)])
def test_parts_each_at_a_power_of_its_own(powers):
    """Parts of uneven small weights, the large one among them, and a row's last part of a few logits."""
    rng = np.random.default_rng(int(powers[1]))
    rows, vocab = len(DRAWS), 8192 * 9 + 11
    x = (-math.log(2.0) * (rng.uniform(*powers, (rows, 10)).repeat(8192, 1)[:, :vocab] + rng.uniform(0, 3, (rows, vocab)))).astype(np.float32)
    x[np.arange(rows), rng.integers(0, vocab, rows)] = 0.0
    x[4, -1] = 0.0
    for kw in (dict(), dict(top_k=1), dict(top_k=30000), dict(top_k=vocab - 1), dict(min_p=1e-13)):
        say("sample", powers, kw)
        check_near(x, DRAWS, **kw)


@pytest.mark.parametrize("powers", [43.0, 44.0, 47.0, 52.0])
@pytest.mark.parametrize("place", [77, 600000, (1 << 20) - 1])
def test_longest_row(place, powers):
    """128 parts, weights in 2^-42: the large one in the first, in between and in the last."""
    rows, vocab = len(DRAWS), 1 << 20
    x = np.full((rows, vocab), np.float32(-math.log(2.0) * powers), np.float32)
    x[:, place] = 0.0
    say("sample", place, powers)
    ids = check_near(x, DRAWS, 42)
    if place >= 8192:   # 8192 of 2^-52 are 8 units
        assert ids[:3] == [0, 0, 0]
    if place < vocab - 8192:
        assert ids[-2:] == [vocab - 1] * 2
    check_near(x, DRAWS, 42, top_k=5)


def test_low_temperatures_and_random_draws():
    """Ordinary logits at low temperatures: most parts lie tens of powers of two below the largest."""
    rng = np.random.default_rng(8)
    x = (rng.standard_normal((32, 100000)) * 2).astype(np.float32)
    x[np.arange(32), rng.integers(0, 100000, 32)] += np.float32(6)
    u = rng.random(32).astype(np.float32)
    u[::4], u[1::4] = 0.0, 1.0
    for heat in (0.02, 0.05, 0.1, 0.2, 0.4):
        for kw in (dict(), dict(top_k=50), dict(top_p=0.95)):
            say("sample", heat, kw)
            check_near(x, u, temperature=heat, **kw)
