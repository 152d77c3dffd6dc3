"""wq_kv_write and wq_kv_read against the oracle, bit for bit.

Coding a row is a fixed sequence of single-precision operations (butterflies,
min and max, one division each for the scale, the zero and every code), which
the oracle repeats in numpy's single precision, so codes, scales, zeros and
the rows read back have one right value.  Every width, head size and page
size; slots in any order, skipped slots; strided rows; and nothing outside
the named slots may change."""

import numpy as np
import pytest
import torch

import dequant_gemv_rht_amd as dq
from oracle import kvcache as OK

from gpu_util import dev, host_f16_bits, say
from kv_util import device_cache, guarded, random_cache

pytestmark = pytest.mark.gpu


def _expect_write(host, x, slots, page, heads, d, bits):
    """The oracle's write of rows x[which] fp16 [tokens][heads][d] into copies of host's arrays."""
    out = {n: None if a is None else a.copy() for n, a in host.items()}
    capacity = host["k"].shape[0] * page
    for which in "kv":
        r = x[which].astype(np.float32) if host["signs"] is None else OK.rotate_rows_f32(x[which], host["signs"])
        if bits == 16:
            codes = r.astype(np.float16)
        else:
            codes, s, z = OK.code_rows(r, bits)
        pl = OK.places(which, bits, d, page)
        for i, slot in enumerate(slots):
            if not 0 <= slot < capacity:
                continue
            p, t = divmod(int(slot), page)
            u = codes[i]
            if bits == 4:
                u = u[:, 0::2] | (u[:, 1::2] << 4)
            out[which][p][:, pl[t]] = u
            if bits != 16:
                out[which + "_params"][p, :, t, 0] = s[i]
                out[which + "_params"][p, :, t, 1] = z[i]
    return out


def _expect_read(host, slots, page, heads, d, bits):
    capacity = host["k"].shape[0] * page
    out = {}
    for which in "kv":
        codes = OK.unpack_pages(which, host[which], bits, d, page).astype(np.float32)
        scale = np.ones(codes.shape[:-1], np.float32)
        if bits != 16:
            scale = host[which + "_params"][..., 0].astype(np.float32)
            codes = codes - host[which + "_params"][..., 1:].astype(np.float32)
        y, sc = np.zeros((len(slots), heads, d), np.float32), np.zeros((len(slots), heads), np.float32)
        for i, slot in enumerate(slots):
            if 0 <= slot < capacity:
                y[i], sc[i] = codes[slot // page, :, slot % page], scale[slot // page, :, slot % page]
        if host["signs"] is not None:
            y = OK.unrotate_rows_f32(y, host["signs"], None if bits == 16 else sc)
        elif bits != 16:
            y = y * sc[..., None]
        out[which] = y.astype(np.float16).reshape(len(slots), -1)
    return out


def _compare_cache(cache, want, label):
    for n in ("k", "v", "k_params", "v_params"):
        if want[n] is None:
            continue
        # equal values; a zero's sign is not part of the definition
        a, b = getattr(cache, n).cpu().numpy(), want[n]
        assert np.array_equal(a, b), f"{label}: {n} differs in {np.sum(a != b)} of {a.size} places"


def _compare_rows(got, want, label):
    g, w = got.cpu().numpy(), want
    assert np.array_equal(g, w), f"{label}: {np.sum(g != w)} of {g.size} values differ"


CASES = [(bits, d, page, rot) for bits in (4, 8, 16) for d in (64, 128, 256) for page in (16, 64)
         for rot in ((False, True) if d >= 128 else (False,))]


@pytest.mark.parametrize("bits,d,page,rot", CASES)
@pytest.mark.parametrize("heads", [1, 3])
def test_write_and_read(bits, d, page, rot, heads):
    say(f"kv write/read bits={bits} d={d} page={page} rotated={rot} heads={heads}")
    rng = np.random.default_rng(bits * 1000 + d + page + heads + rot)
    pages, cols = 5, heads * d
    host, cache = random_cache(rng, pages, page, heads, d, bits, rot)
    capacity = pages * page
    # runs that start anywhere in a quad, single tokens, tokens to skip
    slots = np.concatenate([np.arange(page - 3, 2 * page + 1), rng.permutation(np.arange(3 * page, capacity))[:7],
                            [-1, capacity, np.iinfo(np.int32).max, np.iinfo(np.int32).min, 0]]).astype(np.int32)
    n = len(slots)
    x = {w: (rng.standard_normal((n, heads, d)) * rng.choice([1e-3, 1.0, 30.0], (n, heads, 1))).astype(np.float16)
         for w in "kv"}
    x["k"][0] = 0.0                                 # a row of zeros: scale 1
    x["v"][1] = np.float16(3.0)                     # one value: zero at an end
    x["k"][2, :, 0] = np.float16(65504.0)           # the largest finite values
    x["k"][2, :, 1] = np.float16(-65504.0)
    x["v"][3] = np.float16(6e-8)                    # subnormal: the scale rounds to 0, so 1
    args, bufs = [], []
    for w, ld in (("k", cols + 8), ("v", cols + 64)):
        view, buf = guarded(n, cols, ld)
        view.copy_(torch.from_numpy(x[w].reshape(n, cols)))
        args.append(view)
        bufs.append(buf)
    dq.wq_kv_write(cache, args[0], args[1], dev(slots))
    want = _expect_write(host, x, slots, page, heads, d, bits)
    _compare_cache(cache, want, "write")
    read_slots = np.concatenate([slots, rng.integers(0, capacity, 9)]).astype(np.int32)
    back = _expect_read(want, read_slots, page, heads, d, bits)
    k, v = dq.wq_kv_read(cache, dev(read_slots))
    _compare_rows(k, back["k"], "read k")
    _compare_rows(v, back["v"], "read v")
    # strided outputs: columns past the rows stay as they were
    (ko, kb), (vo, vb) = guarded(len(read_slots), cols, cols + 8), guarded(len(read_slots), cols, cols + 24)
    dq.wq_kv_read(cache, dev(read_slots), out=(ko, vo))
    assert torch.equal(ko, k) and torch.equal(vo, v)
    for buf in (kb, vb):
        assert torch.isnan(buf[0]).all() and torch.isnan(buf[-1]).all() and torch.isnan(buf[1:-1, cols:]).all()


@pytest.mark.parametrize("tokens", [1, 2, 3, 4, 5, 15, 16, 17, 63, 130])
@pytest.mark.parametrize("bits", [4, 8])
def test_write_lengths_and_starts(tokens, bits):
    say(f"kv write tokens={tokens} bits={bits}")
    rng = np.random.default_rng(tokens + bits)
    heads, d, page = 2, 128, 32
    for start in (0, 1, 2, 3, 13, 29):
        host, cache = random_cache(rng, 6, page, heads, d, bits, True)
        order = rng.permutation(6)
        at = start + np.arange(tokens)
        slots = (order[at // page] * page + at % page).astype(np.int32)
        x = {w: rng.standard_normal((tokens, heads, d)).astype(np.float16) for w in "kv"}
        dq.wq_kv_write(cache, dev(x["k"].reshape(tokens, -1)), dev(x["v"].reshape(tokens, -1)), dev(slots))
        _compare_cache(cache, _expect_write(host, x, slots, page, heads, d, bits), f"start {start}")


def test_descending_and_interleaved_slots():
    say("kv write: descending and interleaved slots")
    rng = np.random.default_rng(9)
    heads, d, page = 2, 128, 16
    host, cache = random_cache(rng, 4, page, heads, d, 8)
    up = np.arange(64)
    for slots in (up[::-1], np.stack([up[:32], up[32:]], 1).ravel(), np.concatenate([up[1::2], up[0::2]])):
        slots = slots.astype(np.int32)
        x = {w: rng.standard_normal((64, heads, d)).astype(np.float16) for w in "kv"}
        dq.wq_kv_write(cache, dev(x["k"].reshape(64, -1)), dev(x["v"].reshape(64, -1)), dev(slots))
        host = _expect_write(host, x, slots, page, heads, d, 8)
        _compare_cache(cache, host, "slots")


def test_non_finite_rows_stay_alone():
    say("kv write: rows with infinities and NaN")
    rng = np.random.default_rng(10)
    heads, d, page = 2, 128, 16
    for bits in (4, 8):
        host, cache = random_cache(rng, 2, page, heads, d, bits, True)
        x = {w: rng.standard_normal((8, heads, d)).astype(np.float16) for w in "kv"}
        bad = {w: x[w].copy() for w in "kv"}
        bad["k"][1, 0, 5] = np.nan
        bad["v"][2, 1, 7] = np.inf
        bad["k"][3, 1, 9] = -np.inf
        slots = np.arange(8, dtype=np.int32)
        dq.wq_kv_write(cache, dev(bad["k"].reshape(8, -1)), dev(bad["v"].reshape(8, -1)), dev(slots))
        want = _expect_write(host, x, slots, page, heads, d, bits)
        k, v = (t.view(8, heads, d).cpu().numpy() for t in dq.wq_kv_read(cache, dev(slots)))
        back = _expect_read(want, slots, page, heads, d, bits)
        for got, w, rows in ((k, "k", [(1, 0), (3, 1)]), (v, "v", [(2, 1)])):
            keep = np.ones((8, heads), bool)
            for r in rows:
                keep[r] = False
            assert np.array_equal(got[keep], back[w].reshape(8, heads, d)[keep])


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("d,rot", [(64, False), (128, False), (128, True), (256, False)])
def test_ties_and_signed_zeros(bits, d, rot):
    """Quotients half way between codes (scale 1), rows without a positive or
    without a negative value but with zeros of either sign, all zeros, and
    the smallest numbers."""
    rng = np.random.default_rng(bits + d)
    page, heads, qmax = 16, 2, 2 ** bits - 1
    host, cache = random_cache(rng, 3, page, heads, d, bits, rot)
    rows = []
    for low in (0, -3, -qmax // 2, -qmax):
        r = rng.integers(2 * low, 2 * (low + qmax) + 1, d) / 2
        r[[1, d - 1]] = low, low + qmax
        rows.append(r)
    for sign in (1, -1):
        r = sign * np.abs(rng.standard_normal(d))
        r[::3] = 0.0
        r[1::5] = -0.0
        rows.append(r)
        r = np.where(rng.random(d) < 0.5, 0.0, -0.0)
        r[rng.integers(d)] = sign * 0.25
        rows.append(r)
        rows.append(np.full(d, sign * 2.0 ** -24))
    rows += [np.zeros(d), np.full(d, -0.0), np.where(rng.random(d) < 0.5, 0.0, -0.0)]
    n = len(rows)
    x = {w: np.stack([np.stack([rows[i], rows[(i + 5) % n]]) for i in range(n)]).astype(np.float16) for w in "kv"}
    slots = np.arange(3, 3 + n).astype(np.int32)
    dq.wq_kv_write(cache, dev(x["k"].reshape(n, -1)), dev(x["v"].reshape(n, -1)), dev(slots))
    _compare_cache(cache, _expect_write(host, x, slots, page, heads, d, bits), f"ties bits={bits} d={d}")


def test_fp16_rows_pass_through():
    # 16 bits without rotation: every bit pattern but a NaN's payload
    say("kv write/read: fp16 bits")
    x = torch.arange(65536, dtype=torch.int32).to(torch.int16).view(torch.float16).view(512, 128).cuda()
    cache = dq.KVCache.new(32, 16, 1, 128, 16)
    slots = torch.arange(512, dtype=torch.int32, device="cuda")
    dq.wq_kv_write(cache, x, x.flip(0).contiguous(), slots)
    k, v = dq.wq_kv_read(cache, slots)
    for got, want in ((k, x), (v, x.flip(0))):
        nan = torch.isnan(want)
        assert torch.equal(torch.isnan(got), nan)
        assert np.array_equal(host_f16_bits(got)[~nan.cpu().numpy()], host_f16_bits(want.contiguous())[~nan.cpu().numpy()])


def test_no_tokens():
    say("kv write/read: no tokens")
    cache = dq.KVCache.new(2, 16, 2, 64, 8)
    empty = torch.empty((0, 128), dtype=torch.float16, device="cuda")
    none = torch.empty(0, dtype=torch.int32, device="cuda")
    dq.wq_kv_write(cache, empty, empty, none)
    k, v = dq.wq_kv_read(cache, none)
    assert k.shape == v.shape == (0, 128)


def test_far_pages():
    # a cache past 4 GiB an array: offsets need 64 bits
    say("kv write/read: pages past 4 GiB")
    heads, d, page = 8, 128, 64
    pages = (5 << 30) // (heads * d * page)
    k, v = (torch.empty((pages, heads, page * d), dtype=torch.uint8, device="cuda") for _ in range(2))
    kp, vp = (torch.empty((pages, heads, page, 2), dtype=torch.float16, device="cuda") for _ in range(2))
    cache = dq.KVCache(8, d, heads, page, k, v, kp, vp)
    rng = np.random.default_rng(11)
    x = {w: rng.standard_normal((6, heads, d)).astype(np.float16) for w in "kv"}
    far = [0, 1, (pages - 1) * page + 63, (pages - 1) * page + 62, (pages // 2) * page + 5, pages * page - page]
    slots = np.array(far, np.int32)
    dq.wq_kv_write(cache, dev(x["k"].reshape(6, -1)), dev(x["v"].reshape(6, -1)), dev(slots))
    got = dq.wq_kv_read(cache, dev(slots))
    for t, w in zip(got, "kv"):
        q, s, z = OK.code_rows(x[w].astype(np.float32), 8)
        want = ((q.astype(np.float32) - z[..., None].astype(np.float32)) * s[..., None].astype(np.float32))
        assert np.array_equal(t.cpu().numpy(), want.astype(np.float16).reshape(6, -1))


def test_other_stream():
    say("kv write/read on another stream")
    rng = np.random.default_rng(12)
    heads, d, page = 2, 128, 16
    host, cache = random_cache(rng, 4, page, heads, d, 8)
    x = {w: rng.standard_normal((20, heads, d)).astype(np.float16) for w in "kv"}
    slots = rng.permutation(64)[:20].astype(np.int32)
    k, v, sl = dev(x["k"].reshape(20, -1)), dev(x["v"].reshape(20, -1)), dev(slots)
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    with torch.cuda.stream(st):
        dq.wq_kv_write(cache, k, v, sl)
        a, b = dq.wq_kv_read(cache, sl)
    st.synchronize()
    want = _expect_write(host, x, slots, page, heads, d, 8)
    back = _expect_read(want, slots, page, heads, d, 8)
    _compare_rows(a, back["k"], "k")
    _compare_rows(b, back["v"], "v")


def test_device_cache_helper_matches_layout():
    # the test helper's device copy is what the oracle packed
    rng = np.random.default_rng(13)
    host, _ = random_cache(rng, 2, 16, 1, 64, 8)
    assert np.array_equal(device_cache(host, 16, 1, 64, 8).k.cpu().numpy(), host["k"])
