"""wq_attn_decode on rotated caches: queries of any magnitude that fp16 holds.

A rotated query may be sqrt(128) times larger than fp16's largest number and
is in general not an fp16 value, also where the query's own numbers are
subnormal.  The header promises two fp16 parts (22 bits) either way, so the
tolerances are those of test_gpu_attn_decode.py."""

import numpy as np
import pytest

import dequant_gemv_rht_amd as dq
from oracle import hadamard as OH

from gpu_util import dev, say
from kv_util import random_cache
from test_gpu_attn_decode import check, reference

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("bits", [4, 8, 16])
@pytest.mark.parametrize("d", [128, 256])
@pytest.mark.parametrize("group", [4, 12])          # low parts in spare columns; in operands of their own
def test_rotated_queries_of_any_magnitude(bits, d, group):
    say(f"attn query magnitudes bits={bits} d={d} group={group}")
    rng = np.random.default_rng(50 + bits + d + group)
    heads, page, lens = 2, 32, [100, 65]
    host, cache = random_cache(rng, 8, page, heads, d, bits, True)
    table = rng.permutation(8).reshape(2, 4).astype(np.int32)
    n = dev(np.array(lens, np.int32))
    signs = OH.signs_from_bits(host["signs"], heads * d).reshape(heads, 1, d).astype(np.float64)
    x = rng.standard_normal((2, heads, group, d))
    spread = np.abs(x) * signs                          # every channel's sign the rotation's: all in one rotated channel
    for what, q, scale in (("largest", 65504.0 * np.sign(spread), 4e-6),
                           ("one channel", 65504.0 * (np.arange(d) % 128 == 3) * np.ones_like(x), 1.2e-5 / (d // 128)),
                           ("large", np.clip(2e4 * spread, -65504, 65504), 8e-6),
                           ("ordinary", 1.5 * x, d ** -0.5), ("small", 1e-3 * x, 100.0), ("subnormal", 6e-6 * x, 1e4),
                           ("mixed heads", x * 10.0 ** np.linspace(-5, 4, group)[:, None], 1e-5)):
        q = q.astype(np.float16).reshape(2, heads * group, d)
        got = dq.wq_attn_decode(cache, dev(q.reshape(2, -1)), dev(table), n, scale=scale)
        check(got, reference(host, bits, d, page, q, table, lens, scale), f"{what} bits={bits} d={d} group={group}")
