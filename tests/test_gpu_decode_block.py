"""The example's attention block, prompt and decode steps, against the same
chain in 64 bits on the oracle: projections, rotary positions, cache,
attention and output projection.

Tolerance.  With a 16-bit cache every stage rounds to fp16 (the projections'
outputs, the rotated keys and queries, the attention output, the result) and
the inputs of both projections are rounded once rotated: about eight
roundings of 2^-12 relative each on the way, 7e-4 together, and a score moves
by a few times that; 5e-3 leaves room for the softmax.  With 8 bits a key or
value that the two chains hand over 2^-11 apart may fall on another code: a
step is 1/255 of the row's range, 2e-2 of its RMS, for the few per cent of
the values that lie that near a boundary, so 3e-3 of the RMS; 1e-2 in all.
"""

import os
import subprocess
import sys

import numpy as np
import pytest
import torch

import workloads as W
from oracle import kvcache as OK
from oracle import linear as OL
from oracle import rtn as OR

from gpu_util import say

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, os.path.join(ROOT, "examples"))

import decode_block as DB  # noqa: E402

pytestmark = pytest.mark.gpu


class Chain:
    """The block in 64 bits, from the same random numbers."""

    def __init__(self, block, hidden, q_heads, kv_heads, d, bits, rotate, seed):
        rng = np.random.default_rng(seed)
        signs = W.sign_bits(hidden, rng)
        self.w = {}
        for name, k, n in (("q", hidden, q_heads * d), ("k", hidden, kv_heads * d), ("v", hidden, kv_heads * d),
                           ("o", q_heads * d, hidden)):
            w = W.weight(k, n, rng)
            sg = signs if k == hidden and name != "o" else W.sign_bits(k, rng)
            self.w[name] = (*OR.prepare(w, sg, 4), sg)
        self.cache_signs = W.sign_bits(kv_heads * d, rng) if rotate else None
        self.cos, self.sin = block.cos.cpu().numpy(), block.sin.cpu().numpy()
        self.kv, self.heads, self.d, self.bits = [[], []], (q_heads, kv_heads), d, bits

    def project(self, name, x):
        q, s, z, sg = self.w[name]
        return OL.linear(q, s, z, x.astype(np.float16), sg)

    def rope(self, x, heads, pos):
        x = x.reshape(len(pos), heads, self.d)
        return OK.rope(x, self.cos, self.sin, np.asarray(pos)[None], [0] * (self.d // 2), False)

    def stored(self, x):
        """What the cache holds of rows [n][heads][d], rotated where it is."""
        x = x.astype(np.float16)
        r = OK.rotate_rows_f32(x, self.cache_signs) if self.cache_signs is not None else x.astype(np.float32)
        if self.bits == 16:
            return r.astype(np.float16).astype(np.float64)
        q, s, z = OK.code_rows(r, self.bits)
        return (q.astype(np.float64) - z[..., None]) * s[..., None].astype(np.float64)

    def rows(self, x, pos):
        kvh = self.heads[1]
        k = self.rope(self.project("k", x), kvh, pos)
        v = self.project("v", x).reshape(len(pos), kvh, self.d)
        return self.stored(k), self.stored(v)

    def attend(self, x, k, v):
        """One token x [1][hidden] at position len(k) - 1 over rows k, v [n][kv_heads][d]."""
        qh, kvh = self.heads
        n = len(k)
        q = self.rope(self.project("q", x), qh, [n - 1])
        rot = None if self.cache_signs is None else OK.rotation(self.cache_signs, kvh, self.d)
        page = lambda r: r.transpose(1, 0, 2)[None]   # noqa: E731  one page of n tokens
        y = OK.attend(q, page(k), page(v), np.zeros((1, n), np.int64), [n], self.d ** -0.5, rot=rot)
        return self.project("o", y.reshape(1, -1))


@pytest.mark.parametrize("bits,tol", [(16, 5e-3), (8, 1e-2)])
def test_prompt_and_steps(bits, tol):
    say(f"decode block bits={bits}")
    hidden, qh, kvh, d, seed = 512, 8, 2, 128, 5
    b = DB.AttentionBlock(3, 80, hidden, qh, kvh, d, 4, bits, 16, True, 1e4, seed)
    c = Chain(b, hidden, qh, kvh, d, bits, bits < 16, seed)
    rng = np.random.default_rng(6)
    held = []
    for s, n in enumerate((37, 1, 64)):
        x = rng.standard_normal((n, hidden)).astype(np.float16)
        b.prompt(s, torch.from_numpy(x).cuda())
        held.append(c.rows(x, np.arange(n)))
    for _ in range(4):
        x = rng.standard_normal((3, hidden)).astype(np.float16)
        got = b.step(torch.from_numpy(x).cuda()).float().cpu().numpy()
        for s in range(3):
            n = len(held[s][0])
            new = c.rows(x[s:s + 1], [n])
            held[s] = tuple(np.concatenate([a, r]) for a, r in zip(held[s], new))
            want = c.attend(x[s:s + 1], *held[s])[0]
            rel = np.linalg.norm(got[s] - want) / np.linalg.norm(want)
            say(f"  sequence {s} at {n}: rel-L2 {rel:.2e}")
            assert rel <= tol


@pytest.mark.parametrize("bits,tol", [(16, 5e-3), (8, 1e-2)])
def test_prompt_outputs(bits, tol):
    """Every prompt token's output: attention over itself and the tokens before it."""
    say(f"decode block prompts bits={bits}")
    hidden, qh, kvh, d, seed = 512, 8, 2, 128, 7
    b = DB.AttentionBlock(2, 80, hidden, qh, kvh, d, 4, bits, 16, True, 1e4, seed)
    c = Chain(b, hidden, qh, kvh, d, bits, bits < 16, seed)
    rng = np.random.default_rng(8)
    for s, n in enumerate((1, 53)):
        x = rng.standard_normal((n, hidden)).astype(np.float16)
        got = b.prompt(s, torch.from_numpy(x).cuda()).float().cpu().numpy()
        k, v = c.rows(x, np.arange(n))
        for i in range(n):
            want = c.attend(x[i:i + 1], k[:i + 1], v[:i + 1])[0]
            rel = np.linalg.norm(got[i] - want) / np.linalg.norm(want)
            assert rel <= tol, (s, i, rel)


def test_command():
    out = subprocess.run([sys.executable, os.path.join(ROOT, "examples", "decode_block.py"), "--seqs", "2", "--prompt",
                          "70", "--steps", "3", "--bits", "4"], capture_output=True, text=True, timeout=100)
    assert out.returncode == 0, out.stderr[-2000:]
    assert "us a step" in out.stdout
