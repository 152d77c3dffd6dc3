"""wq_sample against the oracle: tokens equal, their log chances within the
rounding of a 32-bit result (2^-23 relative, and 1e-9 for the fp64 sums)."""

import math

import numpy as np
import pytest
import torch

import dequant_gemv_rht_amd as dq
from oracle import serving as O

from gpu_util import dev, say

pytestmark = pytest.mark.gpu


def check(x, u, temperature=None, top_k=None, top_p=None, min_p=None, ld=None):
    """x: [rows][vocab] fp32 or fp16, the settings: per row or None."""
    rows, vocab = x.shape
    f = lambda v, t: None if v is None else dev(np.asarray(np.broadcast_to(v, rows), t).copy())  # noqa: E731
    logits = dev(x)
    if ld:
        wide = torch.full((rows, ld), float("inf"), dtype=logits.dtype, device="cuda")
        wide[:, :vocab] = logits
        logits = wide[:, :vocab]
    ids, logp = dq.wq_sample(logits, f(u, np.float32), f(temperature, np.float32), f(top_k, np.int32),
                             f(top_p, np.float32), f(min_p, np.float32))
    ids, logp = ids.cpu().numpy(), logp.cpu().numpy()
    for r in range(rows):
        kw = {n: v if np.ndim(v) == 0 else np.asarray(v)[r] for n, v in
              (("temperature", temperature), ("top_k", top_k), ("top_p", top_p), ("min_p", min_p)) if v is not None}
        kw = {n: np.float32(v) if n != "top_k" else int(v) for n, v in kw.items()}
        want, lp = O.sample(x[r], np.float32(u if np.ndim(u) == 0 else u[r]), **kw)
        assert ids[r] == want, f"row {r}: token {ids[r]}, {want} expected ({kw})"
        if math.isinf(lp):
            assert logp[r] == lp
        else:
            assert abs(logp[r] - lp) <= abs(lp) * 2.0 ** -23 + 1e-9, f"row {r}: {logp[r]} for {lp}"
    return ids


def logits_of(rng, rows, vocab, spread, half):
    x = (rng.standard_normal((rows, vocab)) * spread).astype(np.float32)
    return x.astype(np.float16) if half else x


SETTINGS = [dict(), dict(temperature=0.0), dict(temperature=0.6), dict(top_k=1), dict(top_k=40), dict(top_p=0.9),
            dict(top_p=0.999), dict(min_p=0.05), dict(temperature=1.3, top_k=300, top_p=0.8, min_p=0.02),
            dict(temperature=5.0, top_p=0.97), dict(temperature=0.05, top_k=7)]


@pytest.mark.parametrize("half", [False, True])
@pytest.mark.parametrize("vocab", [1, 2, 3, 63, 255, 1000, 4097, 32003, 151936])
def test_settings(vocab, half):
    rng = np.random.default_rng(vocab)
    for spread in (0.3, 3.0):
        for kw in SETTINGS:
            rows = 5 if vocab < 5000 else 2
            say("sample", vocab, half, spread, kw)
            check(logits_of(rng, rows, vocab, spread, half), rng.random(rows).astype(np.float32), **kw)


@pytest.mark.parametrize("rows,vocab,half", [(7, 151936, False), (65, 32003, True), (300, 1500, False), (33, 50001, False)])
def test_settings_of_each_row(rows, vocab, half):
    rng = np.random.default_rng(rows)
    x = logits_of(rng, rows, vocab, 2.5, half)
    x[::4] *= np.asarray(3, x.dtype)
    x[1::3, : vocab - 100] = -np.inf
    pick = lambda *v: np.array([v[i] for i in rng.integers(0, len(v), rows)])  # noqa: E731
    check(x, rng.random(rows).astype(np.float32), temperature=pick(0.0, 0.3, 0.7, 1.0, 2.0),
          top_k=pick(0, -5, 1, 20, 500, vocab, 2 ** 31 - 1), top_p=pick(1.0, 0.1, 0.9, 0.99, 2.0, 0.0),
          min_p=pick(0.0, 0.0, 0.1, 1.0, -1.0), ld=vocab + 5)


@pytest.mark.parametrize("value", [0.0, -0.0, 17.0, -3.0, 1e30, -1e30, 1e-40])
def test_all_equal(value):
    """Every border is a whole number of equal weights."""
    n = 9001
    x = np.full((8, n), value, np.float32)
    if value == 0.0:
        x[:, ::2] = -0.0
    u = np.array([0, 0.25, 0.5, 0.75, 0.999, 1 - 2 ** -24, 1 / 3, 2 ** -24], np.float32)
    check(x, u)
    check(x, u, top_k=100)
    check(x, u, top_p=0.5)
    check(x, u, top_p=0.125, top_k=8000)
    check(x, u, min_p=1.0)


def test_borders_of_equal_weights():
    """Four equal ones among nothing: u and p exactly on the borders."""
    x = np.full((9, 5000), -1e4, np.float32)
    x[:, [7, 900, 4096, 4999]] = 2.5
    u = np.array([0, 0.25, 0.5, 0.75, 0.2499999, 0.7499999, 0.9999999, 0.1, 0.6], np.float32)
    for p in (1.0, 0.5, 0.25, 0.75, 0.7500001, 0.0):
        check(x, u, top_p=p)
        check(x, u, top_p=p, top_k=3)


def test_infinities_and_nans():
    inf, nan = np.inf, np.nan
    x = np.full((8, 700), -1.0, np.float32)
    x[0] = -inf
    x[1] = nan
    x[2, 3:] = -inf
    x[3, [5, 300, 650]] = inf
    x[4, ::2] = nan
    x[5] = -3.4e38
    x[6, 10], x[6, 11] = 3.4e38, -3.4e38
    x[7] = np.where(np.arange(700) == 699, -1e38, -inf)
    for kw in SETTINGS:
        check(x, np.full(8, 0.7, np.float32), **kw)
    y = np.where(np.abs(x) > 6e4, np.sign(x) * 6e4, x).astype(np.float16)
    for kw in SETTINGS:
        check(y, np.full(8, 0.3, np.float32), **kw)


def test_odd_settings():
    rng = np.random.default_rng(1)
    x = logits_of(rng, 6, 3000, 2.0, False)
    u = np.array([0.5, math.nan, -3.0, 2.0, 1.0, 0.0], np.float32)
    check(x, u)
    check(x, np.full(6, 0.4, np.float32), temperature=np.array([math.nan, -1.0, math.inf, 1e-30, 1e30, 1e-45]))
    check(x, np.full(6, 0.4, np.float32), top_p=np.array([math.nan, -1.0, math.inf, 1e-30, 1 - 2 ** -24, 1e-45]))
    check(x, np.full(6, 0.4, np.float32), min_p=np.array([math.nan, -1.0, math.inf, 1e-30, 1 - 2 ** -24, 1.0]))


@pytest.mark.parametrize("temperature", [0.02, 0.05, 0.1, 0.15])
def test_low_temperatures(temperature):
    """top-k's last tokens far below the largest, some of them of no weight."""
    rng = np.random.default_rng(6)
    x = logits_of(rng, 24, 40000, 2.0, False)
    x[:, 100:112] += rng.uniform(0, 6, (24, 12)).astype(np.float32)
    for k in (1, 5, 12, 50, 400, 20000):
        check(x, rng.random(24).astype(np.float32), temperature=temperature, top_k=k, top_p=np.float32([1.0, 0.9] * 12))


@pytest.mark.parametrize("powers", [(32.2, 33.0), (31.0, 36.0), (33.0, 43.0), (44.0, 52.0), (60.0, 90.0)])
def test_cuts_among_small_weights(powers):
    """One large weight, 8000 of 2^-31 to 2^-90 in two of the row's parts, cuts among them and the draw on both sides."""
    rng = np.random.default_rng(int(powers[0] * 10))
    x = np.full((4, 20000), -np.inf, np.float32)
    x[:, 9000] = 3.0
    x[:, 3000:7000] = 3.0 - math.log(2.0) * rng.uniform(*powers, (4, 4000))
    x[:, 15000:19000] = 3.0 - math.log(2.0) * rng.uniform(*powers, (4, 4000))
    x[3, 15000:19000] = x[3, 3000]   # equal ones
    u = np.array([0.0, 0.5, 1 - 2.0 ** -15, 1 - 2.0 ** -18], np.float32)
    for kw in (dict(top_k=1), dict(top_k=2), dict(top_k=50), dict(top_k=5000), dict(top_k=8001), dict(top_k=9000),
               dict(top_p=1 - 2.0 ** -24), dict(top_p=1 - 2.0 ** -22), dict(min_p=2.0 ** -33.5), dict(min_p=1e-30),
               dict(top_k=5000, top_p=1 - 2.0 ** -23), dict(top_k=8001, top_p=1 - 2.0 ** -24, min_p=2.0 ** -33),
               dict(top_k=6000, min_p=1e-13)):
        say("sample", powers, kw)
        ids, logp = dq.wq_sample(dev(x), dev(u), **{n: dev(np.full(4, v, np.int32 if n == "top_k" else np.float32))
                                                    for n, v in kw.items()})
        kw = {n: v if n == "top_k" else float(np.float32(v)) for n, v in kw.items()}
        for r, (i, lp) in enumerate(zip(ids.tolist(), logp.tolist())):
            place, w = O.kept(x[r], **kw)
            at = np.flatnonzero(place == i)
            assert len(at) == 1, f"row {r}: token {i} is not kept ({kw})"
            # A weight is off by 2^-34 of itself and half of 2^-44 of the
            # largest at most, so a sum of the n kept by 2^-34 of itself and
            # n 2^-45, and the draw, u of all of them, by as much: the token's
            # share of the sum lies within twice that of the draw.
            off = 2 * (2.0 ** -34 * w.sum() + len(w) * 2.0 ** -45)
            draw, after = float(u[r]) * w.sum(), float(np.cumsum(w)[at[0]])
            assert after - w[at[0]] - off <= draw <= after + off, f"row {r}: {i}, {after - draw} from the draw ({kw})"
            want = math.log(w[at[0]] / w.sum())
            assert abs(lp - want) <= abs(want) * 2.0 ** -23 + 1e-9, f"row {r}: {lp} for {want}"


@pytest.mark.parametrize("gap", [2.0, 5.0, 9.0, 14.0, 18.0])
def test_chances_near_one(gap):
    """A token that is almost all of the sum: its log chance is as exact as the others' sum."""
    rng = np.random.default_rng(int(gap))
    x = rng.uniform(-1, 1, (12, 30000)).astype(np.float32) - 12
    x[:, 5:9] += 12
    x[np.arange(12), rng.integers(0, 30000, 12)] = np.float32(1 + gap)
    u = np.full(12, 0.5, np.float32)
    for kw in (dict(), dict(top_k=1), dict(top_k=3), dict(top_p=0.5), dict(top_p=0.99999), dict(min_p=0.5), dict(top_k=50, min_p=1e-9)):
        ids, logp = dq.wq_sample(dev(x), dev(u), **{n: dev(np.full(12, v, np.int32 if n == "top_k" else np.float32))
                                                    for n, v in kw.items()})
        kw = {n: v if n == "top_k" else float(np.float32(v)) for n, v in kw.items()}
        for r, (i, lp) in enumerate(zip(ids.tolist(), logp.tolist())):
            place, w = O.kept(x[r], **kw)
            at = np.flatnonzero(place == i)[0]
            # The others' sum s is off by 2^-34 of itself and n 2^-45 (a
            # weight: 2^-34 of itself, half of 2^-44 of the largest), ln(1 - s /
            # all) by twice that at most while s is below half of all, and
            # by 2^-33 of itself through all; then the rounding to 32 bits.
            s = w.sum() - w[at] if len(w) > 1 else 0.0
            want = math.log1p(-s / w.sum())
            assert w[at] > s
            assert abs(lp - want) <= 2 * (s * 2.0 ** -34 + (len(w) - 1) * 2.0 ** -45) + abs(want) * (2.0 ** -33 + 2.0 ** -24), \
                f"row {r}: {lp} for {want} ({kw})"
            assert len(w) > 1 or lp == 0


def test_wide_open():
    """Many tokens within a millionth of each other's chance: the borders need the sums' 64 bits."""
    rng = np.random.default_rng(2)
    n = 262144
    x = (rng.standard_normal((6, n)) * 1e-3).astype(np.float32)
    u = rng.random(6).astype(np.float32)
    check(x, u)
    check(x, u, top_p=0.7)
    check(x, u, top_k=200000, top_p=0.99999)


def test_longest():
    n = 1 << 20
    x = np.zeros((2, n), np.float16)
    x[1, -1] = 9
    check(x, np.array([1 - 2 ** -24, 0.999], np.float32))
    check(x, np.array([0.6, 0.3], np.float32), top_k=n - 1, top_p=0.3)


def test_large_and_small_shift():
    """Logits far from zero: the largest is taken off first."""
    rng = np.random.default_rng(4)
    x = logits_of(rng, 4, 20000, 3.0, False)
    for shift in (1000.0, -1000.0, 64.0):
        check(x + np.float32(shift), rng.random(4).astype(np.float32), top_p=0.95, temperature=0.8)


def test_falling_and_rising_rows():
    x = np.stack([np.arange(30000), -np.arange(30000), np.arange(30000) // 100]).astype(np.float32) * 1e-3
    for kw in SETTINGS:
        check(x, np.array([0.3, 0.6, 0.9], np.float32), **kw)


def test_given_outputs_and_no_rows():
    x = dev(np.zeros((3, 10), np.float32))
    out = torch.full((7,), 55, dtype=torch.int32, device="cuda"), torch.full((7,), 5.5, device="cuda")
    ids, logp = dq.wq_sample(x, torch.full((3,), 0.55, device="cuda"), out=(out[0][2:5], out[1][2:5]))
    assert ids.tolist() == [5, 5, 5] and out[0].tolist() == [55, 55, 5, 5, 5, 55, 55]
    assert out[1][[0, 1, 5, 6]].tolist() == [5.5] * 4
    ids, logp = dq.wq_sample(torch.zeros((0, 10), device="cuda"), torch.zeros(0, device="cuda"))
    assert ids.shape == (0,) and logp.shape == (0,)


def test_same_bits_every_time():
    rng = np.random.default_rng(6)
    x = dev(logits_of(rng, 40, 60000, 2.0, False))
    u = dev(rng.random(40).astype(np.float32))
    p = torch.full((40,), 0.93, device="cuda")
    first = dq.wq_sample(x, u, top_p=p)
    for fill in (0, 255):
        ws = torch.full((dq.wq_sample_workspace(40, 60000) + 16,), fill, dtype=torch.uint8, device="cuda")
        again = dq.wq_sample(x, u, top_p=p, workspace=ws)
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])


def test_captured():
    rng = np.random.default_rng(7)
    x = dev(logits_of(rng, 5, 40000, 2.0, False))
    u = torch.zeros(5, device="cuda")
    p = torch.full((5,), 0.9, device="cuda")
    ws = torch.empty(dq.wq_sample_workspace(5, 40000) + 16, dtype=torch.uint8, device="cuda")
    out = torch.empty(5, dtype=torch.int32, device="cuda"), torch.empty(5, device="cuda")
    call = lambda: dq.wq_sample(x, u, top_p=p, workspace=ws, out=out)  # noqa: E731
    call()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    for turn in range(5):
        now = rng.random(5).astype(np.float32)
        x.mul_(1.05)
        u.copy_(dev(now))
        out[0].zero_()
        g.replay()
        torch.cuda.synchronize()
        host = x.cpu().numpy()
        for r in range(5):
            assert out[0][r].item() == O.sample(host[r], now[r], top_p=np.float32(0.9))[0], (turn, r)
