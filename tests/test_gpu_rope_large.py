"""wq_rope over enough tokens that a wave takes four rounds of heads for one
look-up, against the oracle in 64 bits; tolerance as in test_gpu_rope.py."""

import numpy as np
import pytest
import torch

import dequant_gemv_rht_amd as dq
from oracle import kvcache as OK

from gpu_util import dev, say
from kv_util import guarded
from large_cases import ROPE
from test_gpu_rope import check, tables

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("case", ROPE, ids=str)
def test_many_waves(case):
    d, rot, adjacent, axes, heads, tokens = case
    say(f"rope {case}")
    rng = np.random.default_rng(d + rot + heads)
    half, rows = rot // 2, 300
    cos, sin = tables(rows, rot)
    pos = rng.integers(0, rows, (axes, tokens)).astype(np.int32)
    pos[:, ::97] = -1                                        # outside the table: unchanged
    pos[-1, 5] = rows
    axis = rng.integers(0, axes, half).tolist()
    x = rng.standard_normal((tokens, heads, d)).astype(np.float16)
    args, kw = (dev(cos), dev(sin), dev(pos), d), dict(pair_axis=axis, adjacent=adjacent)
    flat = dev(x.reshape(tokens, -1))
    y, = dq.wq_rope([flat], *args, **kw)
    check(y.cpu().numpy().reshape(x.shape), x, OK.rope(x, cos, sin, pos, axis, adjacent), adjacent, half)
    # strided in place beside a second array of fewer heads: the same bits, nothing past the rows
    few = 1 + heads // 3
    a, abuf = guarded(tokens, heads * d, heads * d + 8)
    b, bbuf = guarded(tokens, few * d, few * d + 24)
    a.copy_(flat)
    b.copy_(flat[:, : few * d])
    dq.wq_rope([a, b], *args, out=[a, b], **kw)
    assert torch.equal(a, y) and torch.equal(b, y[:, : few * d])
    for view, buf in ((a, abuf), (b, bbuf)):
        assert torch.isnan(buf[0]).all() and torch.isnan(buf[-1]).all() and torch.isnan(buf[1:-1, view.shape[1]:]).all()
