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
from kv_util import device_cache
from test_gpu_attn_decode import check, reference

pytestmark = pytest.mark.gpu


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
    heads, d, group, page, n = 8, 128, 4, 64, 2048
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
