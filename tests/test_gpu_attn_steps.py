"""wq_attn_decode over runs of many steps: what a wave carries from one step
to the next (its running reference and sums, the keys and values requested
ahead, the page entries).  Enough sequences and heads that the card is full
without splitting, so a workgroup's run is long.  Tolerances: those of
test_gpu_attn_decode.py, whose derivation does not depend on the length."""

import numpy as np
import pytest
import torch

import dequant_gemv_rht_amd as dq
from oracle import kvcache as OK

from gpu_util import dev, say
from kv_util import device_cache, random_cache
from large_cases import JOINS, MASKED, MOVING, SPLIT_STEPS, STEPS, UNWRITTEN
from test_gpu_attn_decode import check, reference

pytestmark = pytest.mark.gpu
POOL = 2048   # tokens of distinct rows that the sequences' tables are dealt from


def lengths(rng, n, most):
    """`n` lengths up to `most`: the longest, one and none among them, odd ones."""
    lens = rng.integers(1, most + 1, n)
    lens[0] = most
    if n > 3:
        lens[1:4] = 1, 0, most - 17
    return lens.astype(np.int32)


def problem(case, seed, distinct):
    """A cache whose pages several sequences share in any order, and `distinct` sequences over it."""
    rng = np.random.default_rng(seed)
    host, cache = random_cache(rng, POOL // case.page, case.page, case.heads, case.d, case.bits, case.rotated)
    table = rng.integers(0, POOL // case.page, (distinct, -(-case.max_len // case.page))).astype(np.int32)
    q = (1.5 * rng.standard_normal((distinct, case.heads * case.group, case.d))).astype(np.float16)
    return rng, host, cache, table, q, lengths(rng, distinct, case.max_len)


def run(cache, case, table, q, lens, rows, **kw):
    """The call over sequences `rows` (repeats) of the problem."""
    return dq.wq_attn_decode(cache, dev(q[rows].reshape(len(rows), -1)), dev(table[rows]), dev(lens[rows]),
                             max_len=case.max_len, window=case.window, **kw)


@pytest.mark.parametrize("case", STEPS + SPLIT_STEPS + JOINS, ids=str)
def test_many_steps(case):
    say(f"attn {case}")
    distinct = min(case.seqs, 5)
    rng, host, cache, table, q, lens = problem(case, 60 + case.bits + case.d + case.group + case.max_len, distinct)
    rows = rng.permutation(np.arange(case.seqs) % distinct)
    got = run(cache, case, table, q, lens, rows)
    want = reference(host, case.bits, case.d, case.page, q, table, lens, case.d ** -0.5, case.window)
    first = np.array([np.flatnonzero(rows == i)[0] for i in range(distinct)])
    check(got[dev(first)], want, str(case))
    assert torch.equal(got, got[dev(first[rows])])      # equal sequences, equal bits, wherever they are in the batch


@pytest.mark.parametrize("bits", [4, 8, 16])
@pytest.mark.parametrize("d,rotated", [(64, False), (128, True), (256, True)])
def test_pages_outside_the_cache_in_later_steps(bits, d, rotated):
    say(f"attn invalid pages, later steps bits={bits} d={d}")
    case = next(c for c in STEPS if (c.bits, c.d, c.rotated) == (bits, d, rotated))
    rng, host, cache, table, q, lens = problem(case, 70 + bits + d, 6)
    lens[1:4] = 650, 600, 699
    bad = np.array([-1, POOL // case.page, 2 ** 31 - 1, -(2 ** 31)], np.int32)
    gone = rng.random(table.shape) < 0.2
    gone[0, : 3 * 128 // case.page] = True               # nothing in the first three steps
    gone[1] = True                                       # nothing at all
    gone[3, 256 // case.page:] = True                    # nothing after the first two
    table[gone] = bad[rng.integers(0, 4, gone.sum())]
    rows = np.arange(case.seqs) % 6
    got = run(cache, case, table, q, lens, rows)[:6]
    check(got, reference(host, bits, d, case.page, q, table, lens, d ** -0.5), "invalid pages")
    assert not got[1].any()


@pytest.mark.parametrize("bits", [4, 8, 16])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("window", [0, 333])
def test_what_is_masked_never_matters_in_later_steps(bits, d, window):
    """Past the lengths and before the window: NaN and infinities.  Pages are
    each sequence's own, so that what one masks no other sees."""
    say(f"attn garbage, later steps bits={bits} d={d} window={window}")
    rng = np.random.default_rng(80 + bits + d + window)
    heads, group, page, seqs, max_len = next((c.heads, c.group, c.page, c.seqs, c.max_len) for c in MASKED
                                             if (c.bits, c.d, c.window) == (bits, d, window))
    lens = np.array([700, 517, 384, 129], np.int32)
    per = -(-max_len // page)
    host, cache = random_cache(rng, 4 * per, page, heads, d, bits)
    table = rng.permutation(4 * per).reshape(4, per).astype(np.int32)
    q = (1.5 * rng.standard_normal((4, heads * group, d))).astype(np.float16)
    rows = np.arange(seqs) % 4
    call = lambda c: dq.wq_attn_decode(c, dev(q[rows].reshape(seqs, -1)), dev(table[rows]), dev(lens[rows]),   # noqa: E731
                                       max_len=max_len, window=window)
    clean = call(cache)
    check(clean[:4], reference(host, bits, d, page, q, table, lens, d ** -0.5, window), "clean")
    hide = np.ones((4 * per, page), bool)
    for b, n in enumerate(lens):
        for t in range(max(0, n - window) if window else 0, n):
            hide[table[b, t // page], t % page] = False
    hide = np.broadcast_to(hide[:, None, :], (4 * per, heads, page))
    junk = np.array([np.nan, np.inf, -np.inf, 65504.0], np.float16)
    for w in "kv":
        x = OK.unpack_pages(w, host[w], bits, d, page)
        x[hide] = junk[rng.integers(0, 4, (hide.sum(), d))] if bits == 16 else rng.integers(0, 1 << bits, (hide.sum(), d))
        host[w] = OK.pack_pages(w, x, bits)
        if bits != 16:
            host[w + "_params"][hide] = junk[rng.integers(0, 4, (hide.sum(), 2))]
    assert torch.equal(call(device_cache(host, page, heads, d, bits)), clean)


@pytest.mark.parametrize("bits", [4, 8, 16])
def test_scores_and_value_scales_move_from_step_to_step(bits):
    """Scores rise by about 40 over 1500 tokens (or fall, in half of the
    heads), values' sizes change 2^20-fold from token to token and with the
    scores' rise against them: the running reference moves in most steps."""
    say(f"attn moving reference bits={bits}")
    rng = np.random.default_rng(90 + bits)
    heads, group, d, page, seqs, n = next((c.heads, c.group, c.d, c.page, c.seqs, c.max_len) for c in MOVING if c.bits == bits)
    pages = -(-n // page)
    at = np.arange(pages * page).reshape(pages, 1, page)
    k = 0.1 * rng.standard_normal((pages, heads, page, d)).astype(np.float32)
    k[..., 0] = at * (40.0 / n)
    size = np.exp2(rng.uniform(-10, 4, (pages, heads, page)) - 6.0 * at / n)
    v = (size[..., None] * rng.standard_normal(k.shape)).astype(np.float32)
    host = {"signs": None}
    for w, x in (("k", k), ("v", v)):
        if bits == 16:
            host[w], host[w + "_params"] = OK.pack_pages(w, x.astype(np.float16), 16), None
        else:
            c, s, z = OK.code_rows(x, bits)
            host[w], host[w + "_params"] = OK.pack_pages(w, c, bits), np.stack([s, z], -1)
    cache = device_cache(host, page, heads, d, bits)
    q = rng.standard_normal((2, heads * group, d)).astype(np.float16)
    q[:, 0::2, 0], q[:, 1::2, 0] = 1.0, -1.0
    table = np.arange(pages, dtype=np.int32)[None].repeat(2, 0)
    lens = np.array([n, n - 333], np.int32)
    rows = np.arange(seqs) % 2
    got = dq.wq_attn_decode(cache, dev(q[rows].reshape(seqs, -1)), dev(table[rows]), dev(lens[rows]), scale=1.0)
    check(got[:2], reference(host, bits, d, page, q, table, lens, 1.0), "moving reference")
    assert torch.equal(got, got[:2].repeat(seqs // 2, 1))


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("part", [1.0, 0.5])
def test_negative_scales(bits, part):
    """Codes from elsewhere: (c, z, s) and (qmax - c, qmax - z, -s) stand for
    the same value.  All rows, or half of them, in the second form, scores
    that rise by about 60: weights far above the running reference show in
    negative products only."""
    say(f"attn negative scales bits={bits} part={part}")
    rng = np.random.default_rng(95 + bits)
    heads, group, d, page, seqs, n = next((c.heads, c.group, c.d, c.page, c.seqs, c.max_len) for c in MOVING if c.bits == bits)
    pages, qmax = -(-n // page), 2 ** bits - 1
    at = np.arange(pages * page).reshape(pages, 1, page)
    k = 0.1 * rng.standard_normal((pages, heads, page, d)).astype(np.float32)
    k[..., 0] = at * (60.0 / n)
    host = {"signs": None}
    for w, x in (("k", k), ("v", rng.standard_normal(k.shape).astype(np.float32))):
        c, s, z = OK.code_rows(x, bits)
        turned = rng.random(s.shape) < part
        c = np.where(turned[..., None], qmax - c, c).astype(np.uint8)
        z, s = np.where(turned, np.float16(qmax) - z, z), np.where(turned, -s, s)
        host[w], host[w + "_params"] = OK.pack_pages(w, c, bits), np.stack([s, z], -1).astype(np.float16)
    cache = device_cache(host, page, heads, d, bits)
    q = rng.standard_normal((1, heads * group, d)).astype(np.float16)
    q[..., 0] = 1.0
    table = np.arange(pages, dtype=np.int32)[None]
    got = dq.wq_attn_decode(cache, dev(q.reshape(1, -1)).repeat(seqs, 1), dev(table).repeat(seqs, 1),
                            torch.full((seqs,), n, dtype=torch.int32, device="cuda"), scale=1.0)
    check(got[:1], reference(host, bits, d, page, q, table, [n], 1.0), "negative scales")
    assert torch.equal(got, got[:1].repeat(seqs, 1))


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("seqs", [64, 32])
def test_many_value_rows_of_scale_zero(bits, seqs):
    """Most rows of a sequence were never written (a cleared page: scale 0,
    score 0), after some of scores near -76 and before one of +25: the
    unwritten rows' weights, near 2^124 of the first reference, must not
    overflow the sum of weights, in a wave (64 sequences: 16 steps) or where
    splits join (32: two splits of 8 steps, the strong token in the second).
    All queries of a sequence have one score (a head that moves the reference
    moves its neighbours'), and scores differ by 1.5 per cent between
    sequences, so some meet every power of two about there."""
    say(f"attn unwritten rows bits={bits} seqs={seqs}")
    rng = np.random.default_rng(40 + bits + seqs)
    heads, d, group, page, n = next((c.heads, c.d, c.group, c.page, c.max_len) for c in UNWRITTEN
                                    if (c.bits, c.seqs) == (bits, seqs))
    k = np.zeros((n // page, heads, page, d), np.float32)
    v = rng.standard_normal(k.shape).astype(np.float32)
    k[..., 0] = -76.0
    k[-1, :, page - 5, 0] = 25.0
    host = {"signs": None}
    unwritten = np.ones((n // page, 1, page), bool)
    unwritten[:4] = False                    # the first two steps of every wave
    unwritten[-1, :, page - 5] = False
    for w, x in (("k", k), ("v", v)):
        c, s, z = OK.code_rows(x, bits)
        gone = np.broadcast_to(unwritten, s.shape)
        s[gone], z[gone], c[gone] = 0, 0, 0
        host[w], host[w + "_params"] = OK.pack_pages(w, c, bits), np.stack([s, z], -1)
    q = np.zeros((12, heads * group, d), np.float16)
    q[:, :, 0] = (0.92 + 0.015 * np.arange(12))[:, None]
    table = np.arange(n // page, dtype=np.int32)[None].repeat(12, 0)
    cache = device_cache(host, page, heads, d, bits)
    want = reference(host, bits, d, page, q, table, [n] * 12, 1.0)
    rows = np.arange(seqs) % 12
    got = dq.wq_attn_decode(cache, dev(q[rows].reshape(seqs, -1)), dev(table[rows]),
                            torch.full((seqs,), n, dtype=torch.int32, device="cuda"), scale=1.0)
    check(got, want[rows], "unwritten rows")
