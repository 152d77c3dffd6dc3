"""wq_sample about the border of the logits that its bins take, 2^13 powers of
two: rows with parts on both sides of it, against the oracle."""

import math

import numpy as np
import pytest

from gpu_util import say
from test_gpu_sample import check

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kw", [dict(), dict(top_k=1), dict(top_k=40), dict(top_p=0.9), dict(min_p=0.05),
                                dict(top_k=3000, top_p=0.8, min_p=1e-6)])
@pytest.mark.parametrize("temperature", [0.01, 0.05, 1.0, 3.0])
@pytest.mark.parametrize("border", [-8192.0, 8192.0])
def test_parts_on_both_sides(border, temperature, kw):
    """The largest of each part a little above or below the border, in turn."""
    rng = np.random.default_rng(int(temperature * 100))
    power = math.log(2.0) * float(np.float32(temperature))
    vocab = 3 * 8192 + 500
    tops = border + np.array([[0.4, -0.3, -0.2, 0.1], [-0.3, 0.4, -0.1, -0.2], [-0.2, -0.3, -0.1, -0.4], [0.1, 0.2, 0.3, 0.4],
                              [-0.3, -0.2, -0.1, 0.2], [20.0, -0.5, -3.0, -9.0], [-63.0, -1.0, -2.0, -30.0], [62.0, -1.0, 0.5, 61.0]])
    x = (tops.repeat(8192, 1)[:, :vocab] - 6 - 30 * rng.random((8, vocab))) * power
    for part in range(4):
        at = 8192 * part + rng.integers(0, 500, 8)
        x[np.arange(8), at] = tops[:, part] * power
    say("sample", border, temperature, kw)
    check(x.astype(np.float32), rng.random(8).astype(np.float32), temperature=temperature, **kw)


def test_two_tokens():
    """A chance of 0.27 below the border is drawn."""
    x = np.full((4, 10000), -400.0, np.float32)
    x[:, 7], x[:, 8201] = -283.90, -283.92
    assert check(x, np.array([0.1, 0.5, 0.7, 0.9], np.float32), temperature=0.05).tolist() == [7, 7, 8201, 8201]
