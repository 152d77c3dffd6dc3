"""wq_lora against the oracle, within the bound of its 32-bit sums (derived in
oracle/serving.py) and half a step of the output's type: one row to many, one
adapter to one a row, rows without one, every rank step, odd widths, strided
rows, rows of large and of no magnitude, in place, several linears at once."""

import numpy as np
import pytest
import torch

import dequant_gemv_rht_amd as dq
from oracle import serving as O

from gpu_util import dev, say

pytestmark = pytest.mark.gpu


def make(rng, count, rank, k, n, m, f32=False, x_scale=1.0):
    a = (rng.standard_normal((count, rank, k)) / np.sqrt(k)).astype(np.float16)
    b = (rng.standard_normal((count, n, rank)) * 0.2).astype(np.float16)
    x = (rng.standard_normal((m, k)) * x_scale).astype(np.float16)
    base = rng.standard_normal((m, n)).astype(np.float32 if f32 else np.float16)
    return a, b, x, base


def check(y, want, off, f32, what):
    y = y.float().cpu().numpy().astype(np.float64)
    step = np.abs(want) * (2.0 ** -24 if f32 else 2.0 ** -11) + (0 if f32 else 2.0 ** -25)
    bad = ~(np.abs(y - want) <= off + step * (1 + 2.0 ** -10))
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size} off, first at {np.argwhere(bad)[0]}, " \
                          f"{y[bad][0]} for {want[bad][0]} +- {(off + step)[bad][0]}"


def ids_of(kind, rng, m, count):
    if kind == "each":
        return rng.permutation(m) % count
    if kind == "one":
        return np.full(m, count - 1)
    if kind == "runs":
        return np.sort(rng.integers(0, count, m))
    if kind == "some":
        return np.where(rng.random(m) < 0.4, rng.choice([-1, count, -2 ** 31, 2 ** 31 - 1], m), rng.integers(0, count, m))
    return np.full(m, -1)


CASES = [   # m, count, rank, k, n, ids
    (1, 1, 8, 128, 1, "one"), (1, 3, 16, 2560, 1024, "one"), (2, 5, 24, 256, 77, "each"), (7, 7, 16, 1024, 512, "each"),
    (16, 4, 32, 640, 130, "runs"), (17, 3, 16, 512, 129, "some"), (33, 2, 64, 384, 65, "some"), (64, 64, 16, 256, 96, "each"),
    (64, 1, 128, 1280, 200, "one"), (65, 9, 40, 256, 33, "some"), (100, 6, 104, 128, 64, "runs"), (255, 31, 8, 128, 63, "some"),
    (256, 256, 8, 128, 48, "each"), (257, 200, 16, 128, 50, "each"), (300, 2, 16, 256, 100, "some"),
    (300, 300, 8, 128, 24, "each"), (513, 4, 64, 512, 72, "runs"), (700, 5, 48, 128, 31, "some"), (20, 3, 16, 128, 40, "none"),
    (3, 2, 8, 9728, 2560, "each"), (1000, 3, 16, 1152, 16, "runs"),
]


@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("m,count,rank,k,n,kind", CASES)
def test_against_oracle(m, count, rank, k, n, kind, f32):
    rng = np.random.default_rng(m * 1000 + rank)
    a, b, x, base = make(rng, count, rank, k, n, m, f32)
    scales = rng.uniform(0.25, 2.0, count).astype(np.float32)
    ids = ids_of(kind, rng, m, count).astype(np.int32)
    say("lora", m, count, rank, k, n, kind, f32)
    (y,) = dq.wq_lora([dev(a)], [dev(b)], [dev(x)], dev(ids), [dev(base)], scales=dev(scales))
    want, off = O.lora(a, b, x, ids, base, scales)
    check(y, want, off, f32, "y")
    out = (ids < 0) | (ids >= count)
    assert np.array_equal(y.cpu().numpy()[out], base[out])   # bit for bit


@pytest.mark.parametrize("kind", ["each", "runs", "some"])
@pytest.mark.parametrize("count", [8, 9, 40])
@pytest.mark.parametrize("m", [31, 32, 33, 129, 256, 257, 1025])
def test_few_and_many_adapters(m, count, kind):
    """Rows on both sides of where the groups are made in another way."""
    rng = np.random.default_rng(m * 100 + count)
    a, b, x, base = make(rng, count, 72, 384, 70, m)
    ids = ids_of(kind, rng, m, count).astype(np.int32)
    say("lora", m, count, kind)
    (y,) = dq.wq_lora([dev(a)], [dev(b)], [dev(x)], dev(ids), [dev(base)])
    check(y, *O.lora(a, b, x, ids, base), False, "y")


@pytest.mark.parametrize("m,count,rank", [(2047, 3, 16), (2048, 3, 16), (2049, 40, 72), (2500, 300, 128), (4097, 2, 24)])
def test_many_rows(m, count, rank):
    rng = np.random.default_rng(m)
    ids = ids_of("runs" if count < 10 else "some", rng, m, count).astype(np.int32)
    a, b, xs, bases, want = [], [], [], [], []
    x = None
    for n, f32 in ((300, False), (33, True), (512, False)):
        A, B, X, base = make(rng, count, rank, 256, n, m, f32)
        x = X if x is None else x
        a.append(dev(A)), b.append(dev(B)), xs.append(dev(x)), bases.append(dev(base))
        want.append((O.lora(A, B, x, ids, base), f32))
    for y, (w, f32) in zip(dq.wq_lora(a, b, xs, dev(ids), bases), want):
        check(y, *w, f32, "y")


def test_several_linears_strides_and_in_place():
    rng = np.random.default_rng(5)
    m, count = 37, 4
    ids = ids_of("some", rng, m, count).astype(np.int32)
    shapes = [(8, 256, 96, False), (16, 256, 33, True), (64, 128, 200, False), (16, 640, 1, False), (24, 128, 8, True),
              (128, 128, 130, False), (8, 128, 15, False), (32, 256, 64, True)]
    a, b, xs, bases, want, ys, bufs = [], [], [], [], [], [], []
    scales = rng.uniform(-1, 1, count).astype(np.float32)
    for rank, k, n, f32 in shapes:
        A, B, X, base = make(rng, count, rank, k, n, m, f32)
        want.append(O.lora(A, B, X, ids, base, scales))
        wide = torch.full((m, k + 24), float("nan"), dtype=torch.float16, device="cuda")
        wide[:, 8:8 + k] = dev(X)
        buf = torch.full((m + 2, n + 8), 7.0, dtype=torch.float32 if f32 else torch.float16, device="cuda")
        view = buf.view(-1)[16: 16 + m * (n + 5)].view(m, n + 5)[:, :n]   # rows of odd alignment
        view.copy_(dev(base))
        bufs.append((buf, buf.clone(), view))
        a.append(dev(A)), b.append(dev(B)), xs.append(wide[:, 8:8 + k]), bases.append(view)
    fresh = dq.wq_lora(a, b, xs, dev(ids), bases, scales=dev(scales))
    ys = dq.wq_lora(a, b, xs, dev(ids), bases, scales=dev(scales), out=bases)
    for i, (rank, k, n, f32) in enumerate(shapes):
        check(ys[i], *want[i], f32, f"linear {i}")
        assert torch.equal(fresh[i], ys[i]) and ys[i].data_ptr() == bases[i].data_ptr()
        buf, before, view = bufs[i]
        view.copy_(before.view(-1)[16: 16 + m * (n + 5)].view(m, n + 5)[:, :n])
        assert torch.equal(buf, before)   # nothing beside the rows was written


@pytest.mark.parametrize("m", [3, 50, 300])
def test_columns_of_one_wide_array_in_place(m):
    rng = np.random.default_rng(m)
    count, k, widths = 5, 256, (96, 32, 32)
    ids = ids_of("some", rng, m, count).astype(np.int32)
    wide = torch.full((m, sum(widths) + 8), 5.0, dtype=torch.float16, device="cuda")
    parts, a, b, want, at = [], [], [], [], 0
    x = None
    for n in widths:
        A, B, X, base = make(rng, count, 16, k, n, m)
        x = X if x is None else x
        view = wide[:, at:at + n]
        view.copy_(dev(base))
        parts.append(view), a.append(dev(A)), b.append(dev(B))
        want.append(O.lora(A, B, x, ids, base))
        at += n
    xs = [dev(x)] * 3
    ys = dq.wq_lora(a, b, xs, dev(ids), parts, out=parts)
    for y, w in zip(ys, want):
        check(y, *w, False, "y")
    assert (wide[:, at:] == 5.0).all()


@pytest.mark.parametrize("m,kind", [(5, "each"), (40, "some"), (300, "runs")])
@pytest.mark.parametrize("x_scale", [1e-6, 60.0, 3000.0])
def test_magnitudes(m, kind, x_scale):
    """A x far above fp16's range and far below it."""
    rng = np.random.default_rng(int(x_scale) + m)
    a, b, x, base = make(rng, 3, 16, 256, 40, m, True, x_scale)
    a = (a.astype(np.float32) * (200.0 if x_scale > 1 else 1e-2)).astype(np.float16)
    x[m // 2] = 0
    ids = ids_of(kind, rng, m, 3).astype(np.int32)
    say("lora magnitudes", m, kind, x_scale)
    (y,) = dq.wq_lora([dev(a)], [dev(b)], [dev(x)], dev(ids), [dev(base)])
    check(y, *O.lora(a, b, x, ids, base), True, "y")


@pytest.mark.parametrize("m", [6, 70, 300])
def test_infinities_and_nans_stay_in_their_row(m):
    rng = np.random.default_rng(m)
    a, b, x, base = make(rng, 2, 16, 128, 50, m)
    ids = ids_of("each", rng, m, 2).astype(np.int32)
    bad = [1, m - 2]
    x[1, 5], x[m - 2, 127], base[3, 7] = np.inf, np.nan, np.inf
    (y,) = dq.wq_lora([dev(a)], [dev(b)], [dev(x)], dev(ids), [dev(base)])
    good = np.ones(m, bool)
    good[bad] = False
    with np.errstate(all="ignore"):
        want, off = O.lora(a, b, np.where(np.isfinite(x), x, 0), ids, np.where(np.isfinite(base), base, 0))
    y = y.float().cpu().numpy()
    assert not np.isfinite(y[bad]).any() and y[3, 7] == np.inf
    y[3, 7], good_rows = want[3, 7], np.flatnonzero(good)
    check(torch.from_numpy(y[good_rows]), want[good_rows], off[good_rows], False, "other rows")


def test_unused_adapters_are_not_met():
    """Adapters that no row names may hold anything."""
    rng = np.random.default_rng(8)
    a, b, x, base = make(rng, 4, 16, 128, 50, 20)
    ids = np.where(np.arange(20) % 2, 3, 1).astype(np.int32)
    want, off = O.lora(a, b, x, ids, base)
    a[[0, 2]], b[[0, 2]] = np.nan, np.inf
    (y,) = dq.wq_lora([dev(a)], [dev(b)], [dev(x)], dev(ids), [dev(base)])
    check(y, want, off, False, "y")


def test_no_rows():
    rng = np.random.default_rng(8)
    a, b, x, base = make(rng, 4, 16, 128, 50, 0)
    (y,) = dq.wq_lora([dev(a)], [dev(b)], [dev(x)], dev(np.zeros(0, np.int32)), [dev(base)])
    assert y.shape == (0, 50)


@pytest.mark.parametrize("m", [1, 12, 64, 500])
def test_same_bits_every_time_and_any_workspace(m):
    rng = np.random.default_rng(m)
    a, b, x, base = (dev(v) for v in make(rng, 5, 24, 640, 200, m))
    ids = dev(ids_of("some", rng, m, 5).astype(np.int32))
    bytes_ = dq.wq_lora_workspace([a], [b], m)
    ys = []
    for fill in (0, 255):
        ws = torch.full((bytes_,), fill, dtype=torch.uint8, device="cuda")
        ys.append(dq.wq_lora([a], [b], [x], ids, [base], workspace=ws)[0])
    ys.append(dq.wq_lora([a], [b], [x], ids, [base])[0])
    assert torch.equal(ys[0], ys[1]) and torch.equal(ys[0], ys[2])


def test_captured():
    rng = np.random.default_rng(4)
    a, b, x, base = make(rng, 3, 16, 256, 70, 24)
    ids = dev(np.zeros(24, np.int32))
    d = [dev(v) for v in (a, b, x, base)]
    ws = torch.empty(dq.wq_lora_workspace([d[0]], [d[1]], 24), dtype=torch.uint8, device="cuda")
    out = torch.empty_like(d[3])
    call = lambda: dq.wq_lora([d[0]], [d[1]], [d[2]], ids, [d[3]], workspace=ws, out=[out])  # noqa: E731
    call()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    for turn in range(5):   # the rows' adapters change from replay to replay
        now = ids_of("some", rng, 24, 3).astype(np.int32)
        ids.copy_(dev(now))
        out.zero_()
        g.replay()
        torch.cuda.synchronize()
        check(out, *O.lora(a, b, x, now, base), False, f"replay {turn}")
