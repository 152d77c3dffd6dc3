"""wq_kv_write and wq_kv_read over enough rows that a wave takes a span of
several quads of tokens: against the oracle, bit for bit, as in
test_gpu_kvcache.py.  Slots come in runs of every length from 1 on, which
start and end anywhere in a quad, in a span and in a page, with skipped tokens
between them and inside them."""

import numpy as np
import pytest
import torch

import dequant_gemv_rht_amd as dq

from gpu_util import dev, say
from kv_util import guarded, random_cache
from large_cases import ROWS
from test_gpu_kvcache import _compare_cache, _compare_rows, _expect_read, _expect_write

pytestmark = pytest.mark.gpu


def scattered_slots(rng, tokens, capacity):
    """`tokens` slots: the cache cut into runs, dealt in any order; some skipped."""
    cuts = np.cumsum(rng.choice([1, 1, 2, 3, 4, 5, 7, 8, 16, 17, 33, 64, 150], capacity))
    runs = np.split(np.arange(capacity), cuts[cuts < capacity])
    slots = np.concatenate([runs[i] for i in rng.permutation(len(runs))])[:tokens].astype(np.int32)
    gone = rng.random(tokens) < 0.02
    gone[[0, 15, 16, 31, 32, tokens - 1]] = True     # at the spans' borders
    slots[gone] = rng.choice([-1, capacity, 2 ** 31 - 1, -(2 ** 31)], gone.sum())
    return slots


@pytest.mark.parametrize("case", ROWS, ids=str)
def test_spans_of_several_quads(case):
    bits, d, rot, heads, tokens, page = case
    say(f"kv rows {case}")
    rng = np.random.default_rng(bits * 1000 + d + heads + rot)
    pages, cols = -(-(tokens + 500) // page), heads * d
    host, cache = random_cache(rng, pages, page, heads, d, bits, rot)
    capacity = pages * page
    rng2 = np.random.default_rng(1)
    for slots in (scattered_slots(rng, tokens, capacity), (3 + np.arange(tokens)).astype(np.int32)):
        x = {w: (rng2.standard_normal((tokens, heads, d)) * rng2.choice([1e-3, 1.0, 30.0], (tokens, heads, 1)))
             .astype(np.float16) for w in "kv"}
        args = []
        for w, ld in (("k", cols + 8), ("v", cols + 64)):
            view, _ = guarded(tokens, cols, ld)
            view.copy_(torch.from_numpy(x[w].reshape(tokens, cols)))
            args.append(view)
        dq.wq_kv_write(cache, args[0], args[1], dev(slots))
        host = _expect_write(host, x, slots, page, heads, d, bits)
        _compare_cache(cache, host, "write")
        back = _expect_read(host, slots, page, heads, d, bits)
        (ko, kb), (vo, vb) = guarded(tokens, cols, cols + 8), guarded(tokens, cols, cols + 24)
        dq.wq_kv_read(cache, dev(slots), out=(ko, vo))
        _compare_rows(ko, back["k"], "read k")
        _compare_rows(vo, back["v"], "read v")
        for buf in (kb, vb):
            assert torch.isnan(buf[0]).all() and torch.isnan(buf[-1]).all() and torch.isnan(buf[1:-1, cols:]).all()
