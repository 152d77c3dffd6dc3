"""Pins of the key-value cache oracle: the layouts place every element once,
the coding rule on rows worked by hand, attention against a direct sum and
its empty rows, rotary positions against complex multiplication (CPU only)."""

import numpy as np
import pytest

from oracle import kvcache as OK
from oracle.hadamard import rht, rht_inverse


@pytest.mark.parametrize("which", ["k", "v"])
@pytest.mark.parametrize("bits", [4, 8, 16])
@pytest.mark.parametrize("d,page", [(64, 16), (128, 32), (256, 16)])
def test_every_element_has_one_place(which, bits, d, page):
    p = OK.places(which, bits, d, page)
    assert sorted(p.ravel().tolist()) == list(range(page * OK.units(bits, d)))


def test_places_by_hand():
    # keys, 8 bits, 128 channels: panels of 64 bytes over 16 tokens
    assert OK.key_place(0, 63, 8, 128) == 63
    assert OK.key_place(1, 0, 8, 128) == 64
    assert OK.key_place(0, 64, 8, 128) == 1024
    assert OK.key_place(17, 65, 8, 128) == 2048 + 1024 + 64 + 1
    # 4 bits, 64 channels: 32-byte rows, one panel; fp16: panels of 32 values
    assert OK.key_place(3, 5, 4, 64) == 3 * 32 + 5
    assert OK.key_place(2, 40, 16, 64) == 16 * 32 + 2 * 32 + 8
    # values: the four tokens of a quad side by side
    assert [OK.value_place(t, 7, 8, 128) for t in (0, 1, 3, 4)] == [28, 29, 31, 512 + 28]


@pytest.mark.parametrize("bits", [4, 8, 16])
def test_pack_round_trip(bits):
    rng = np.random.default_rng(1)
    c = rng.integers(0, 16 if bits == 4 else 256, (3, 2, 16, 64))
    c = c.astype(np.float16 if bits == 16 else np.uint8)
    for which in "kv":
        arr = OK.pack_pages(which, c, bits)
        assert np.array_equal(OK.unpack_pages(which, arr, bits, 64, 16), c)
    if bits == 4:   # even channel in the low half
        one = np.zeros((1, 1, 16, 64), np.uint8)
        one[0, 0, 0, 1] = 9
        assert OK.pack_pages("k", one, 4)[0, 0, 0] == 0x90


def test_code_rows_by_hand():
    q, s, z = OK.code_rows(np.array([[-1.0, 0.0, 0.5, 2.0]], np.float32), 4)
    assert s[0] == np.float16(0.2) and z[0] == 5 and q.tolist() == [[0, 5, 8, 15]]   # 7.5 to even: 8
    q, s, z = OK.code_rows(np.zeros((1, 4), np.float32), 8)
    assert s[0] == 1 and z[0] == 0 and q.tolist() == [[0, 0, 0, 0]]
    # zero is always in the range: a row of one sign has its zero at an end
    q, s, z = OK.code_rows(np.array([[10.0, 12.0]], np.float32), 8)
    assert z[0] == 0 and q[0, 1] == 255
    q, s, z = OK.code_rows(np.array([[-10.0, -12.0]], np.float32), 8)
    assert z[0] == 255 and q[0, 1] == 0


def test_rotation_is_the_hadamard_oracles():
    rng = np.random.default_rng(2)
    signs = rng.integers(0, 1 << 32, 2 * 256 // 32, dtype=np.uint64).astype(np.uint32)
    x = rng.standard_normal((3, 2, 256)).astype(np.float16)
    r = OK.rotation(signs, 2, 256)
    want = rht(x.reshape(3, 512).astype(np.float64), signs).reshape(3, 2, 256)
    assert np.allclose(np.einsum("hij,thj->thi", r, x.astype(np.float64)), want, atol=1e-12)
    assert np.allclose(OK.rotate_rows_f32(x, signs), want, atol=1e-5)
    back = rht_inverse(want.reshape(3, 512), signs).reshape(3, 2, 256)
    assert np.allclose(OK.unrotate_rows_f32(want.astype(np.float32), signs), back, atol=1e-5)
    codes, scale = rng.integers(-15, 16, (3, 2, 256)).astype(np.float32), rng.uniform(0.1, 1, (3, 2)).astype(np.float16)
    vals = codes.astype(np.float64) * scale[..., None]
    assert np.allclose(OK.unrotate_rows_f32(codes, signs, scale),
                       rht_inverse(vals.reshape(3, 512), signs).reshape(3, 2, 256), atol=1e-5)


def test_attend_direct():
    rng = np.random.default_rng(3)
    pages, kvh, page, d = 4, 2, 16, 64
    k, v = rng.standard_normal((2, pages, kvh, page, d))
    q = rng.standard_normal((2, 4, d))
    table = np.array([[2, 0], [3, 9]])
    y = OK.attend(q, k, v, table, [18, 20], 0.125)
    # sequence 0, query head 3 -> key-value head 1: pages 2, then 0
    kk = np.concatenate([k[2, 1], k[0, 1, :2]])
    vv = np.concatenate([v[2, 1], v[0, 1, :2]])
    w = np.exp(kk @ q[0, 3] * 0.125)
    assert np.allclose(y[0, 3], (w[:, None] * vv).sum(0) / w.sum())
    # sequence 1: page 9 does not exist, so only page 3's 16 tokens count
    w = np.exp(k[3, 0] @ q[1, 0] * 0.125)
    assert np.allclose(y[1, 0], (w[:, None] * v[3, 0]).sum(0) / w.sum())
    # the last 3 positions; nothing at all
    y = OK.attend(q, k, v, table, [18, 0], 0.125, window=3)
    kk, vv = np.concatenate([k[2, 0, 15:], k[0, 0, :2]]), np.concatenate([v[2, 0, 15:], v[0, 0, :2]])
    w = np.exp(kk @ q[0, 1] * 0.125)
    assert np.allclose(y[0, 1], (w[:, None] * vv).sum(0) / w.sum())
    assert not y[1].any()


def test_attend_rotation_cancels():
    # rotated keys and values with a rotated query: the unrotated result
    rng = np.random.default_rng(4)
    k, v = rng.standard_normal((2, 1, 2, 16, 128))
    q = rng.standard_normal((1, 4, 128))
    signs = rng.integers(0, 1 << 32, 8, dtype=np.uint64).astype(np.uint32)
    r = OK.rotation(signs, 2, 128)
    rk, rv = (np.einsum("hij,phtj->phti", r, x) for x in (k, v))
    a = OK.attend(q, k, v, [[0]], [11], 0.1)
    b = OK.attend(q, rk, rv, [[0]], [11], 0.1, rot=r)
    assert np.allclose(a, b, atol=1e-12)


@pytest.mark.parametrize("adjacent", [False, True])
def test_rope_is_a_complex_product(adjacent):
    rng = np.random.default_rng(5)
    x = rng.standard_normal((2, 3, 24))
    angle = rng.uniform(0, 6, (10, 8))
    cos, sin = np.cos(angle), np.sin(angle)
    pos = np.array([[4, 10], [9, 1]])
    axis = [0, 1, 1, 0, 0, 0, 1, 0]
    y = OK.rope(x, cos, sin, pos, axis, adjacent)
    for i in range(8):
        a, b = (2 * i, 2 * i + 1) if adjacent else (i, i + 8)
        for t in range(2):
            p = pos[axis[i], t]
            w = np.exp(1j * angle[p, i]) if p < 10 else 1.0
            z = (x[t, :, a] + 1j * x[t, :, b]) * w
            assert np.allclose(y[t, :, a], z.real) and np.allclose(y[t, :, b], z.imag)
    assert np.array_equal(y[..., 16:], x[..., 16:])
