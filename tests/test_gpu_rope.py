"""wq_rope against the oracle in 64 bits.

a c - b s is two products and a sum in fp32 (error below 3 x 2^-24 of |a| +
|b|) and one rounding to fp16 (2^-11 of the result, 2^-25 below the normal
range): |error| <= 2^-11 |y| + 2^-22 (|a| + |b|) + 2^-25."""

import numpy as np
import pytest
import torch

import dequant_gemv_rht_amd as dq
from oracle import kvcache as OK

from gpu_util import dev, say
from kv_util import guarded

pytestmark = pytest.mark.gpu


def tables(rows, rot, base=10000.0):
    angle = np.arange(rows)[:, None] * base ** (-np.arange(0, rot, 2) / rot)
    return np.cos(angle).astype(np.float32), np.sin(angle).astype(np.float32)


def check(got, x, want, adjacent, half):
    g, w = got.astype(np.float64), want
    y = np.abs(x.astype(np.float64))
    size = np.zeros_like(y)
    for i in range(half):
        a, b = (2 * i, 2 * i + 1) if adjacent else (i, i + half)
        size[..., a] = size[..., b] = y[..., a] + y[..., b]
    assert (np.abs(g - w) <= 2.0 ** -11 * np.abs(w) + 2.0 ** -22 * size + 2.0 ** -25).all()
    assert np.array_equal(got[..., 2 * half:], x[..., 2 * half:])


@pytest.mark.parametrize("d,rot", [(64, 64), (64, 16), (128, 128), (128, 96), (256, 256), (256, 64), (80, 32), (8 * 13, 48)])
@pytest.mark.parametrize("adjacent", [False, True])
@pytest.mark.parametrize("axes", [1, 2, 3, 4])
def test_rope(d, rot, adjacent, axes):
    say(f"rope d={d} rot={rot} adjacent={adjacent} axes={axes}")
    rng = np.random.default_rng(d + rot + axes)
    half, rows = rot // 2, 50
    cos, sin = tables(rows, rot)
    for tokens, heads in ((1, (1,)), (3, (4, 2)), (37, (5, 1, 3))):
        pos = rng.integers(0, rows, (axes, tokens)).astype(np.int32)
        pos[-1, -1] = [-1, rows, 2 ** 31 - 1, -(2 ** 31)][axes - 1]   # outside the table: unchanged
        axis = {0: [i * axes // half for i in range(half)], 1: [i % axes for i in range(half)],
                2: rng.integers(0, axes, half).tolist()}[tokens % 3]
        xs = [rng.standard_normal((tokens, h, d)).astype(np.float16) for h in heads]
        want = [OK.rope(x, cos, sin, pos, axis, adjacent) for x in xs]
        args = dev(cos), dev(sin), dev(pos), d
        kw = dict(pair_axis=axis if axes > 1 else None, adjacent=adjacent)
        flat = [dev(x.reshape(tokens, -1)) for x in xs]
        got = dq.wq_rope(flat, *args, **kw)
        for g, x, w in zip(got, xs, want):
            check(g.cpu().numpy().reshape(x.shape), x, w, adjacent, half)
        # strided in place: the same bits, nothing past the rows
        views = [guarded(tokens, x.shape[1] * d, x.shape[1] * d + 8 * (i + 1)) for i, x in enumerate(xs)]
        for (view, _), f in zip(views, flat):
            view.copy_(f)
        dq.wq_rope([v for v, _ in views], *args, out=[v for v, _ in views], **kw)
        for (view, buf), g in zip(views, got):
            assert torch.equal(view, g)
            assert torch.isnan(buf[0]).all() and torch.isnan(buf[-1]).all() and torch.isnan(buf[1:-1, view.shape[1]:]).all()


def test_far_positions_and_many_tokens():
    say("rope far positions")
    rng = np.random.default_rng(3)
    cos, sin = tables(200000, 128, 1e6)
    pos = rng.integers(0, 200000, 3001).astype(np.int32)
    x = rng.standard_normal((3001, 10, 128)).astype(np.float16)
    y, = dq.wq_rope([dev(x.reshape(3001, -1))], dev(cos), dev(sin), dev(pos), 128)
    check(y.cpu().numpy().reshape(x.shape), x, OK.rope(x, cos, sin, pos[None], [0] * 64, False), False, 64)


def test_no_tokens():
    y, = dq.wq_rope([torch.empty((0, 128), dtype=torch.float16, device="cuda")], torch.ones((4, 32), device="cuda"),
                    torch.ones((4, 32), device="cuda"), torch.empty(0, dtype=torch.int32, device="cuda"), 64)
    assert y.shape == (0, 128)
