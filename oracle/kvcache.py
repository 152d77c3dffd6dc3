"""Paged key-value cache, attention of one new token, rotary positions (oracle).

Test infrastructure only: see the package docstring for who may use it.

The cache format is the library's own (include/wq.h): rows of integer codes
with one scale and zero each ([W01] paragraph on group-wise affine integer
quantisation, one group per row) or fp16 values, optionally behind the
block-128 random Hadamard rotation ([W01] paragraph on the random Hadamard
transform).  Every element is placed and fetched by its own index formula.
"""

from __future__ import annotations

import numpy as np

from .hadamard import hadamard, signs_from_bits


def units(bits: int, d: int) -> int:
    return d // 2 if bits == 4 else d


def key_place(t: int, u: int, bits: int, d: int) -> int:
    """Unit u of the page's token t in a page and head of the key array."""
    n = units(bits, d)
    p = min(n, 32 if bits == 16 else 64)
    return (t // 16) * 16 * n + (u // p) * 16 * p + (t % 16) * p + u % p


def value_place(t: int, u: int, bits: int, d: int) -> int:
    return (t // 4) * 4 * units(bits, d) + 4 * u + t % 4


def places(which: str, bits: int, d: int, page: int) -> np.ndarray:
    """[page][units] places of every row's units."""
    f = key_place if which == "k" else value_place
    return np.array([[f(t, u, bits, d) for u in range(units(bits, d))] for t in range(page)])


def pack_pages(which, codes, bits):
    """Codes (or fp16 values) [pages][heads][page][d] -> the array [pages][heads][page * units]."""
    pages, heads, page, d = codes.shape
    if bits == 4:
        u = (codes[..., 0::2] | (codes[..., 1::2] << 4)).astype(np.uint8)
    else:
        u = codes.astype(np.float16 if bits == 16 else np.uint8)
    out = np.empty((pages, heads, page * units(bits, d)), u.dtype)
    out[:, :, places(which, bits, d, page)] = u
    return out


def unpack_pages(which, arr, bits, d, page):
    """Inverse of pack_pages."""
    u = arr[:, :, places(which, bits, d, page)]
    if bits != 4:
        return u
    return np.stack([u & 15, u >> 4], -1).reshape(*u.shape[:-1], d)


def dequant_pages(which, arr, params, bits, d, page):
    """fp64 values [pages][heads][page][d]."""
    c = unpack_pages(which, arr, bits, d, page).astype(np.float64)
    if bits == 16:
        return c
    par = params.astype(np.float64)
    return (c - par[..., 1:]) * par[..., :1]


def rotation(signs, heads: int, d: int) -> np.ndarray:
    """R of every head, fp64 [heads][d][d]: H D / sqrt(128) per block of 128."""
    sg = signs_from_bits(signs, heads * d).astype(np.float64).reshape(heads, d)
    h = hadamard(128).astype(np.float64) / np.sqrt(128.0)
    m = np.zeros((d, d))
    for b in range(0, d, 128):
        m[b:b + 128, b:b + 128] = h
    return m[None] * sg[:, None, :]


def _hadamard_f32(x):
    """Seven butterfly stages in fp32, then 1/sqrt(128) rounded to fp32: the library's order of operations."""
    shape = x.shape
    x = x.reshape(-1, 128).astype(np.float32)
    h = 1
    while h < 128:
        y = x.reshape(-1, 128 // (2 * h), 2, h)
        x = np.stack([y[:, :, 0] + y[:, :, 1], y[:, :, 0] - y[:, :, 1]], 2).reshape(-1, 128)
        h *= 2
    return (x * np.float32(0.08838834764831845)).reshape(shape)


def rotate_rows_f32(x, signs):
    """R x in single precision, x fp16 [tokens][heads][d]."""
    _, heads, d = x.shape
    sg = signs_from_bits(signs, heads * d).astype(np.float32).reshape(heads, d)
    return _hadamard_f32(x.astype(np.float32) * sg)


def unrotate_rows_f32(x, signs, scale=None):
    """R^T x in single precision.  Coded rows: x is code - zero, whose
    transform is a whole number (exact), and scale [tokens][heads] their
    scales, each times 1/sqrt(128) and rounded before the one product."""
    _, heads, d = x.shape
    sg = signs_from_bits(signs, heads * d).astype(np.float32).reshape(heads, d)
    if scale is None:
        return _hadamard_f32(x) * sg
    h = hadamard(128).astype(np.float64)
    y = (x.astype(np.float64).reshape(-1, d // 128, 128) @ h).reshape(x.shape).astype(np.float32)
    return y * (scale.astype(np.float32) * np.float32(0.08838834764831845))[..., None] * sg


def code_rows(x, bits):
    """The rule of wq_kv_write in single precision: fp32 [...][d] -> (codes, scale fp16, zero fp16)."""
    f = np.float32
    x = x.astype(f)
    qmax = f((1 << bits) - 1)
    lo = np.minimum(x.min(-1), f(0))
    hi = np.maximum(x.max(-1), f(0))
    with np.errstate(over="ignore"):
        s = np.minimum((hi - lo) / qmax, f(65504)).astype(np.float16)
    s = np.where(s == 0, np.float16(1), s)
    sf = s.astype(f)
    z = np.clip(np.rint((f(0) - lo) / sf), f(0), qmax)   # never -0
    q = np.clip(np.rint(x / sf[..., None] + z[..., None]), f(0), qmax)
    return q.astype(np.uint8), s, z.astype(np.float16)


def attend(q, keys, values, table, lens, scale, window=0, rot=None):
    """fp64 [seqs][q_heads][d].  q [seqs][q_heads][d]; keys, values fp64
    [pages][kv_heads][page][d] as stored; rot: rotation(...) or None."""
    seqs, qh, d = q.shape
    pages, kvh, page, _ = keys.shape
    out = np.zeros((seqs, qh, d))
    for b in range(seqs):
        n = int(lens[b])
        pos = np.arange(max(0, n - window) if window else 0, max(n, 0))
        pg = np.asarray(table)[b, pos // page].astype(np.int64)
        ok = (pg >= 0) & (pg < pages)
        pos, pg = pos[ok], pg[ok]
        if len(pos) == 0:
            continue
        for h in range(qh):
            g = h // (qh // kvh)
            x = q[b, h].astype(np.float64)
            if rot is not None:
                x = rot[g] @ x
            s = keys[pg, g, pos % page] @ x * scale
            p = np.exp(s - s.max())
            y = (p / p.sum()) @ values[pg, g, pos % page]
            out[b, h] = rot[g].T @ y if rot is not None else y
    return out


def rope(x, cos, sin, positions, pair_axis, adjacent):
    """fp64 [tokens][heads][d]; positions [axes][tokens]."""
    y = x.astype(np.float64).copy()
    half = cos.shape[1]
    for i in range(half):
        a, b = (2 * i, 2 * i + 1) if adjacent else (i, i + half)
        p = np.asarray(positions)[pair_axis[i]]
        ok = (p >= 0) & (p < cos.shape[0])
        c = np.where(ok, cos[np.where(ok, p, 0), i].astype(np.float64), 1.0)[:, None]
        s = np.where(ok, sin[np.where(ok, p, 0), i].astype(np.float64), 0.0)[:, None]
        u, v = y[:, :, a].copy(), y[:, :, b].copy()
        y[:, :, a], y[:, :, b] = u * c - v * s, v * c + u * s
    return y
