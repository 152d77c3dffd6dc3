"""wq_attn_decode against the oracle's attention in 64 bits, on the same coded
cache.

Tolerance.  The cache's values are exact in the kernel (codes less an integer
zero are whole numbers, scales are applied in fp32); what rounds is
 * the query, to fp16 once rotated: 2^-11 relative per channel at most, so a
   score of magnitude a few moves by a few 2^-12 and a weight by as much,
 * the softmax weights, to fp16: 2^-11 relative at most each,
 * the output, to fp16: 2^-11.
Each is relative to the term it rounds and independent over the terms, so the
relative error of a whole output is at most about (2^-10 + 2^-11) / sqrt(3) +
2^-12 ~ 1.1e-3; one row of 64 to 256 channels may exceed that by chance, by
less than a factor 2.5.  A single value of 5 RMS may meet all three roundings
at their largest: 5 x 2 x 2^-10 = 1e-2 of the RMS.  Hence rel-L2 <= 1.5e-3
over all outputs, 3e-3 for each (sequence, head), max-abs <= 1e-2 x that
row's RMS.
"""

import numpy as np
import pytest
import torch

import dequant_gemv_rht_amd as dq
from oracle import kvcache as OK

from gpu_util import dev, say
from kv_util import device_cache, guarded, random_cache, values

pytestmark = pytest.mark.gpu

ALL, ROW, MAX = 1.5e-3, 3e-3, 1e-2


def check(got, want, label):
    g = got.float().cpu().numpy().astype(np.float64).reshape(want.shape)
    assert np.isfinite(g).all(), f"{label}: non-finite output"
    d = g - want
    n = np.linalg.norm(want)
    rel = np.linalg.norm(d) / n if n else np.linalg.norm(d)
    rn = np.linalg.norm(want, axis=-1)
    row = np.where(rn > 0, np.linalg.norm(d, axis=-1) / np.where(rn > 0, rn, 1), np.linalg.norm(d, axis=-1))
    rms = rn / np.sqrt(want.shape[-1])
    mx = (np.abs(d).max(-1) / np.where(rms > 0, rms, 1)).max()
    say(f"  {label}: rel-L2 {rel:.2e}, worst row {row.max():.2e}, max/rms {mx:.2e}")
    assert rel <= ALL and row.max() <= ROW and mx <= MAX, f"{label}: {rel:.3e} {row.max():.3e} {mx:.3e}"


def problem(rng, bits, d, heads, group, page, lens, rotated=False, q_scale=1.5, spare=2, extra_cols=0):
    seqs = len(lens)
    per = max(1, -(-max(max(lens), 1) // page))
    pages = seqs * per + spare
    host, cache = random_cache(rng, pages, page, heads, d, bits, rotated)
    table = rng.permutation(pages)[: seqs * per].reshape(seqs, per).astype(np.int32)
    if extra_cols:
        table = np.concatenate([table, np.full((seqs, extra_cols), 1 << 30, np.int32)], 1)
    q = (q_scale * rng.standard_normal((seqs, heads * group, d))).astype(np.float16)
    return host, cache, table, q


def reference(host, bits, d, page, q, table, lens, scale, window=0):
    heads = host["k"].shape[1]
    rot = None if host["signs"] is None else OK.rotation(host["signs"], heads, d)
    return OK.attend(q, values(host, "k", bits, d, page), values(host, "v", bits, d, page), table, lens, scale,
                     window, rot)


def run_case(seed, bits, d, heads, group, page, lens, rotated=False, window=0, **kw):
    rng = np.random.default_rng(seed)
    host, cache, table, q = problem(rng, bits, d, heads, group, page, lens, rotated, **kw)
    got = dq.wq_attn_decode(cache, dev(q.reshape(len(lens), -1)), dev(table), dev(np.array(lens, np.int32)),
                            max_len=max(lens), window=window)
    want = reference(host, bits, d, page, q, table, lens, d ** -0.5, window)
    check(got, want, f"bits={bits} d={d} heads={heads}x{group} page={page} window={window}")


LENS = [1, 2, 15, 16, 17, 31, 33, 100, 255]


@pytest.mark.parametrize("bits", [4, 8, 16])
@pytest.mark.parametrize("d,rotated", [(64, False), (128, False), (128, True), (256, False), (256, True)])
@pytest.mark.parametrize("page", [16, 32, 128])
def test_formats(bits, d, rotated, page):
    say(f"attn formats bits={bits} d={d} rotated={rotated} page={page}")
    run_case(bits + d + page + rotated, bits, d, 2, 4, page, LENS, rotated)


@pytest.mark.parametrize("heads,group", [(1, 1), (8, 1), (3, 2), (2, 5), (1, 7), (4, 8), (1, 16), (1, 17), (2, 20), (1, 40)])
@pytest.mark.parametrize("bits", [4, 8, 16])
def test_head_layouts(heads, group, bits):
    say(f"attn heads={heads} group={group} bits={bits}")
    run_case(heads * 100 + group, bits, 128, heads, group, 16, [5, 64, 130], bits != 16)


@pytest.mark.parametrize("length", [127, 128, 129, 511, 512, 513, 1023, 1025, 2047, 2049, 4096, 5000])
@pytest.mark.parametrize("bits", [4, 8])
def test_long_lengths(length, bits):
    # one sequence: split over workgroups and joined
    say(f"attn length={length} bits={bits}")
    run_case(length + bits, bits, 128, 2, 4, 64, [length], True)


def test_ragged_long():
    say("attn ragged")
    run_case(77, 8, 128, 2, 4, 32, [3000, 1, 700, 0, 1500, 64, 2999, 16], True)
    run_case(78, 4, 64, 2, 2, 16, [2500, 1, 700, 0, 1500], False)
    run_case(79, 16, 256, 1, 4, 16, [1700, 3, 0, 900], True)


@pytest.mark.parametrize("window", [1, 2, 15, 16, 17, 100, 500, 1999, 2000, 5000])
def test_window(window):
    say(f"attn window={window}")
    run_case(window, 8, 128, 2, 4, 16, [1, 20, 2000, 517, 0], True, window=window)
    run_case(window + 1, 16, 64, 2, 2, 64, [1, 20, 1100, 517, 0], False, window=window)


def test_empty_rows_are_zero():
    say("attn empty rows")
    rng = np.random.default_rng(5)
    host, cache, table, q = problem(rng, 8, 128, 2, 4, 16, [40, 40, 40])
    lens = np.array([0, -5, 7], np.int32)
    out, buf = guarded(3, 1024, 1032)
    dq.wq_attn_decode(cache, dev(q.reshape(3, -1)), dev(table), dev(lens), max_len=40, out=out)
    assert not out[:2].any() and out[2].any()
    assert torch.isnan(buf[0]).all() and torch.isnan(buf[4]).all() and torch.isnan(buf[1:4, 1024:]).all()
    # no positions at all: an empty table
    y = dq.wq_attn_decode(cache, dev(q.reshape(3, -1)), torch.empty((3, 0), dtype=torch.int32, device="cuda"), dev(lens))
    assert y.shape == (3, 1024) and not y.any()
    y = dq.wq_attn_decode(cache, dev(q.reshape(3, -1))[:0], dev(table)[:0], dev(lens)[:0])
    assert y.shape == (0, 1024)


def test_lengths_above_max_len_count_as_max_len():
    say("attn max_len")
    rng = np.random.default_rng(6)
    host, cache, table, q = problem(rng, 8, 128, 2, 4, 16, [96, 96])
    args = dev(q.reshape(2, -1)), dev(table)
    got = dq.wq_attn_decode(cache, *args, dev(np.array([96, 2 ** 31 - 1], np.int32)), max_len=50)
    check(got, reference(host, 8, 128, 16, q, table, [50, 50], 128 ** -0.5), "clamped")
    got = dq.wq_attn_decode(cache, *args, dev(np.array([96, 13], np.int32)))   # default: what the table holds
    check(got, reference(host, 8, 128, 16, q, table, [96, 13], 128 ** -0.5), "default")


@pytest.mark.parametrize("bits", [4, 8, 16])
@pytest.mark.parametrize("page", [16, 64])
def test_pages_outside_the_cache_take_no_part(bits, page):
    say(f"attn invalid pages bits={bits} page={page}")
    rng = np.random.default_rng(7 + bits + page)
    lens = [5 * page + 3, 4 * page, 2 * page, 9]
    host, cache, table, q = problem(rng, bits, 128, 2, 4, page, lens)
    table[0, 1] = -1
    table[0, 5] = host["k"].shape[0]
    table[1, 0] = 2 ** 31 - 1
    table[2, :] = -(2 ** 31)
    got = dq.wq_attn_decode(cache, dev(q.reshape(4, -1)), dev(table), dev(np.array(lens, np.int32)))
    check(got, reference(host, bits, 128, page, q, table, lens, 128 ** -0.5), "invalid pages")
    assert not got[2].any()


@pytest.mark.parametrize("bits", [4, 8, 16])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_what_is_masked_never_matters(bits, d):
    # everything past the lengths, and before the window, is NaN or infinity
    say(f"attn garbage bits={bits} d={d}")
    rng = np.random.default_rng(8 + bits + d)
    page, lens, window = 32, [1, 37, 64, 70, 200], 50
    host, cache, table, q = problem(rng, bits, d, 2, 4, page, lens)
    clean = dq.wq_attn_decode(cache, dev(q.reshape(5, -1)), dev(table), dev(np.array(lens, np.int32)), window=window)
    seen = np.zeros((host["k"].shape[0], page), bool)
    for b, n in enumerate(lens):
        for t in range(max(0, n - window), n):
            seen[table[b, t // page], t % page] = True
    hide = np.broadcast_to(~seen[:, None, :], (host["k"].shape[0], 2, page))
    junk = np.array([np.nan, np.inf, -np.inf, 65504.0], np.float16)
    for w in "kv":
        if bits == 16:
            x = OK.unpack_pages(w, host[w], 16, d, page)
            x[hide] = junk[rng.integers(0, 4, (hide.sum(), d))]
            host[w] = OK.pack_pages(w, x, 16)
        else:
            x = OK.unpack_pages(w, host[w], bits, d, page)
            x[hide] = rng.integers(0, 1 << bits, (hide.sum(), d))
            host[w] = OK.pack_pages(w, x, bits)
            host[w + "_params"][hide] = junk[rng.integers(0, 4, (hide.sum(), 2))]
    dirty = device_cache(host, page, 2, d, bits)
    got = dq.wq_attn_decode(dirty, dev(q.reshape(5, -1)), dev(table), dev(np.array(lens, np.int32)), window=window)
    assert torch.equal(got, clean)


def test_strides_and_wide_tables():
    say("attn strides")
    rng = np.random.default_rng(9)
    lens = [70, 3, 129]
    host, cache, table, q = problem(rng, 8, 128, 2, 4, 16, lens, True, extra_cols=3)
    view, _ = guarded(3, 1024, 1088)
    view.copy_(torch.from_numpy(q.reshape(3, -1)))
    out, buf = guarded(3, 1024, 2048)
    wide = torch.full((3, table.shape[1] + 5), -7, dtype=torch.int32, device="cuda")
    wide[:, 1:table.shape[1] + 1] = dev(table)
    n = torch.tensor([0, *lens], dtype=torch.int32, device="cuda")[1:]   # 4-byte aligned only
    y = dq.wq_attn_decode(cache, view, wide[:, 1:table.shape[1] + 1], n, max_len=129, out=out)
    assert y.data_ptr() == out.data_ptr()
    check(out, reference(host, 8, 128, 16, q, table, lens, 128 ** -0.5), "strided")
    assert torch.isnan(buf[1:4, 1024:]).all() and torch.isnan(buf[0]).all()


@pytest.mark.parametrize("bits", [4, 8, 16])
def test_value_scales_far_apart(bits):
    # a peaked softmax whose strongest token has tiny values, and a long tail
    # of weights near 2^-17 whose values are large: the tail must keep its
    # precision (fp16 weights alone would lose it)
    say(f"attn value scales bits={bits}")
    rng = np.random.default_rng(10 + bits)
    d, page, n = 128, 64, 4000
    pages = -(-n // page)
    k = np.zeros((pages, 1, page, d), np.float32)
    k[..., 0] = 1.0
    k[0, 0, 5, 0] = 13.0
    v = (100.0 * rng.standard_normal((pages, 1, page, d)) + 50.0).astype(np.float32)
    v[0, 0, 5] = 1e-3 * rng.standard_normal(d)
    host = {"signs": None}
    for w, x in (("k", k), ("v", v)):
        if bits == 16:
            host[w], host[w + "_params"] = OK.pack_pages(w, x.astype(np.float16), 16), None
        else:
            c, s, z = OK.code_rows(x, bits)
            host[w], host[w + "_params"] = OK.pack_pages(w, c, bits), np.stack([s, z], -1)
    q = np.zeros((1, 4, d), np.float16)
    q[0, :, 0] = [1.0, 0.5, 1.3, 0.0]
    table = rng.permutation(pages).reshape(1, -1).astype(np.int32)
    inv = np.argsort(table[0])
    for w in "kv":   # page 0 of the arrays holds token 5, wherever it sits in the sequence
        assert host[w].shape[0] == pages and len(inv) == pages
    cache = device_cache(host, page, 1, d, bits)
    got = dq.wq_attn_decode(cache, dev(q.reshape(1, -1)), dev(table), dev(np.array([n], np.int32)), scale=1.0)
    check(got, reference(host, bits, d, page, q, table, [n], 1.0), "scales")


@pytest.mark.parametrize("bits", [4, 8])
def test_value_scales_of_zero(bits):
    """Rows of scale 0 are zeros, whatever their weights: alone in a sequence,
    in all of it, and in the tokens of the largest scores (spread over some
    hundred powers of two) among others.  Where such a token takes all the
    weight the output is nearly 0, so errors are taken against the values'
    own size, 1."""
    d, heads, group, page = 128, 2, 4, 16
    rng = np.random.default_rng(23)
    lens = [1, 5, 33, 200, 300, 129]
    host, cache, table, q = problem(rng, bits, d, heads, group, page, lens, q_scale=60.0)
    k = values(host, "k", bits, d, page)
    zero = host["v_params"]
    for b, n in enumerate(lens):
        for h in range(heads):
            if b < 2:
                gone = range(n)
            else:
                rows = np.stack([k[table[b, t // page], h, t % page] for t in range(n)])
                top = (q[b, h * group:(h + 1) * group].astype(np.float64) @ rows.T).argsort(-1)
                gone = {int(t) for r in top[: 2] for t in r[-3:]}   # half of the heads
            for t in gone:
                zero[table[b, t // page], h, t % page, 0] = 0
    cache = device_cache(host, page, heads, d, bits)
    got = dq.wq_attn_decode(cache, dev(q.reshape(len(lens), -1)), dev(table), dev(np.array(lens, np.int32)))
    want = reference(host, bits, d, page, q, table, lens, d ** -0.5)
    g = got.float().cpu().numpy().astype(np.float64).reshape(want.shape)
    assert np.isfinite(g).all() and not g[:2].any()
    assert np.abs(g - want).max() <= MAX * np.abs(values(host, "v", bits, d, page)).max()


def test_large_scores():
    # scores of several hundred: the softmax is one token, no overflow
    say("attn large scores")
    run_case(21, 8, 128, 2, 4, 16, [300, 40], False, q_scale=100.0)
    run_case(22, 16, 64, 2, 4, 16, [300, 40], False, q_scale=100.0)


def test_tiny_and_huge_values():
    say("attn magnitudes")
    rng = np.random.default_rng(23)
    for scale in (1e-3, 1e3):
        lens = [33, 500]
        host, cache = random_cache(rng, 40, 16, 2, 128, 8, True, channel_scale=scale)
        table = rng.permutation(40)[:64 // 2].reshape(1, 32).repeat(2, 0).astype(np.int32)
        q = (1.0 / scale * rng.standard_normal((2, 8, 128))).astype(np.float16)
        got = dq.wq_attn_decode(cache, dev(q.reshape(2, -1)), dev(table), dev(np.array(lens, np.int32)))
        check(got, reference(host, 8, 128, 16, q, table, lens, 128 ** -0.5), f"scale {scale}")


def test_zeros_at_the_ends_of_the_code_range():
    # rows of one sign: the zero is 0 or qmax and every code far from it
    say("attn one-signed rows")
    rng = np.random.default_rng(24)
    for bits in (4, 8):
        x = np.abs(rng.standard_normal((4, 2, 16, 128))).astype(np.float32) + 4.0
        x[2:] *= -1.0
        host = {"signs": None}
        for w in "kv":
            c, s, z = OK.code_rows(x, bits)
            assert set(np.unique(z)) == {0.0, float(2 ** bits - 1)}
            host[w], host[w + "_params"] = OK.pack_pages(w, c, bits), np.stack([s, z], -1)
        q = rng.standard_normal((1, 8, 128)).astype(np.float16)
        table = np.array([[2, 0, 3, 1]], np.int32)
        cache = device_cache(host, 16, 2, 128, bits)
        got = dq.wq_attn_decode(cache, dev(q.reshape(1, -1)), dev(table), dev(np.array([61], np.int32)))
        check(got, reference(host, bits, 128, 16, q, table, [61], 128 ** -0.5), f"bits={bits}")


def test_shared_pages():
    # two sequences that share a prefix, as drafted tokens of one sequence do
    say("attn shared pages")
    rng = np.random.default_rng(25)
    host, cache, table, q = problem(rng, 8, 128, 2, 4, 16, [90, 90, 90], True)
    table[:] = table[0]
    lens = [88, 89, 90]
    got = dq.wq_attn_decode(cache, dev(q.reshape(3, -1)), dev(table), dev(np.array(lens, np.int32)))
    check(got, reference(host, 8, 128, 16, q, table, lens, 128 ** -0.5), "shared")


def test_far_pages():
    # keys and values past 4 GiB: offsets need 64 bits
    say("attn pages past 4 GiB")
    heads, d, page = 8, 128, 64
    pages = (5 << 30) // (heads * d * page)
    rng = np.random.default_rng(26)
    small, near = random_cache(rng, 4, page, heads, d, 8)
    k, v = (torch.empty((pages, heads, page * d), dtype=torch.uint8, device="cuda") for _ in range(2))
    kp, vp = (torch.empty((pages, heads, page, 2), dtype=torch.float16, device="cuda") for _ in range(2))
    far = [pages - 1, pages // 2, pages - 2, 0]
    for i, p in enumerate(far):
        k[p], v[p], kp[p], vp[p] = near.k[i], near.v[i], near.k_params[i], near.v_params[i]
    q = dev((1.5 * rng.standard_normal((1, 32 * d))).astype(np.float16))
    lens = torch.tensor([250], dtype=torch.int32, device="cuda")
    a = dq.wq_attn_decode(near, q, dev(np.array([[0, 1, 2, 3]], np.int32)), lens)
    b = dq.wq_attn_decode(dq.KVCache(8, d, heads, page, k, v, kp, vp), q, dev(np.array([far], np.int32)), lens)
    assert torch.equal(a, b) and a.any()


def test_workspace_reuse_and_repeats():
    say("attn repeats")
    rng = np.random.default_rng(27)
    lens = [3000, 10, 1200]
    host, cache, table, q = problem(rng, 8, 128, 2, 4, 32, lens, True)
    args = cache, dev(q.reshape(3, -1)), dev(table), dev(np.array(lens, np.int32))
    first = dq.wq_attn_decode(*args)
    need = dq.wq_attn_decode_workspace(cache, 3, 8, table.shape[1] * 32)
    ws = torch.full((max(need, 16),), 255, dtype=torch.uint8, device="cuda")   # NaN everywhere
    for _ in range(3):
        assert torch.equal(dq.wq_attn_decode(*args, workspace=ws), first)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        other = dq.wq_attn_decode(*args)
    st.synchronize()
    assert torch.equal(other, first)


def test_graph_replays():
    say("attn graph")
    rng = np.random.default_rng(28)
    heads, group, d, page = 2, 4, 128, 16
    host, cache, table, q = problem(rng, 8, d, heads, group, page, [900, 900], True)
    k = torch.zeros((2, heads * d), dtype=torch.float16, device="cuda")
    v, qd = torch.zeros_like(k), dev(q.reshape(2, -1))
    slots, lens, tab = torch.zeros(2, dtype=torch.int32, device="cuda"), \
        torch.zeros(2, dtype=torch.int32, device="cuda"), dev(table)
    out = torch.empty_like(qd)
    ws = torch.empty(max(16, dq.wq_attn_decode_workspace(cache, 2, heads * group, 900)), dtype=torch.uint8, device="cuda")

    def step():
        dq.wq_kv_write(cache, k, v, slots)
        dq.wq_attn_decode(cache, qd, tab, lens, max_len=900, workspace=ws, out=out)

    lens.fill_(1)
    slots.copy_(tab[:, 0] * page)
    step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for t in (5, 300, 899):
        pos = torch.tensor([t, t // 2], device="cuda")
        slots.copy_(tab.gather(1, (pos // page)[:, None])[:, 0] * page + pos % page)
        lens.copy_(pos + 1)
        k.normal_()
        v.normal_()
        qd.normal_()
        g.replay()
        got = out.clone()
        torch.cuda.synchronize()
        step()
        assert torch.equal(out, got)
        arrays = {n: getattr(cache, n).cpu().numpy() for n in ("k", "k_params", "v", "v_params")}
        h = dict(arrays, signs=host["signs"])
        want = reference(h, 8, d, page, qd.cpu().numpy().reshape(2, -1, d), table, lens.cpu().numpy(), d ** -0.5)
        check(got, want, f"replay at {t}")
