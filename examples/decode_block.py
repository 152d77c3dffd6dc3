"""The attention side of a decoder block, prompt and decode steps, on the library's calls.

    python examples/decode_block.py [--bits 4|8|16] [--seqs 8] [--prompt 500] [--steps 32]

One block's query, key, value and output projections (int4, rotated), rotary
positions, a paged key-value cache and attention over it.  Weights and
activations are synthetic.  A decode step, or a prompt, is five calls:

    q, k, v = the three projections, one launch      (wq_linear_batch)
    q, k    = rotary positions                       (wq_rope)
    the new keys and values into the cache           (wq_kv_write)
    attention over every sequence's cached tokens    (wq_attn_decode)
    the output projection                            (wq_linear)
"""

import argparse
import os
import sys
import time

import numpy as np
import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import dequant_gemv_rht_amd as dq  # noqa: E402
import workloads as W  # noqa: E402


class AttentionBlock:
    """Projections, cache and page tables of one block for `seqs` sequences of up to `max_len` tokens."""

    def __init__(self, seqs, max_len, hidden=2560, q_heads=32, kv_heads=8, head_dim=128, weight_bits=4, cache_bits=8,
                 page_size=64, rotate_cache=True, base=1e6, seed=0):
        self.seqs, self.max_len, self.head_dim, self.page_size = seqs, max_len, head_dim, page_size
        rng = np.random.default_rng(seed)
        signs = self._words(W.sign_bits(hidden, rng))      # one vector: the three inputs are rotated once
        self.weights = {}
        for name, k, n in (("q", hidden, q_heads * head_dim), ("k", hidden, kv_heads * head_dim),
                           ("v", hidden, kv_heads * head_dim), ("o", q_heads * head_dim, hidden)):
            w = torch.from_numpy(W.weight(k, n, rng)).cuda()
            sg = signs if k == hidden and name != "o" else self._words(W.sign_bits(k, rng))
            self.weights[name] = dq.quantize_weight(w, weight_bits, sg)
        per_seq = -(-max_len // page_size)
        cache_signs = (self._words(W.sign_bits(kv_heads * head_dim, rng))
                       if rotate_cache and cache_bits < 16 and head_dim % 128 == 0 else None)
        self.cache = dq.KVCache.new(seqs * per_seq, page_size, kv_heads, head_dim, cache_bits, cache_signs)
        # pages dealt out in any order; a server hands them out as sequences grow
        order = torch.from_numpy(rng.permutation(seqs * per_seq)).cuda()
        self.table = order.view(seqs, per_seq).to(torch.int32).contiguous()
        self.lens = torch.zeros(seqs, dtype=torch.int32, device="cuda")
        self.longest = 0                                   # known on the host: bounds the attention launch
        angle = (torch.arange(max_len, device="cuda", dtype=torch.float64)[:, None]
                 * base ** (-torch.arange(0, head_dim, 2, device="cuda", dtype=torch.float64) / head_dim))
        self.cos, self.sin = angle.cos().float(), angle.sin().float()

    @staticmethod
    def _words(bits):
        return torch.from_numpy(bits.view(np.int32)).cuda()

    def _qkv(self, x, positions):
        w = self.weights
        q, k, v = dq.wq_linear_batch([w["q"], w["k"], w["v"]], [x, x, x])
        dq.wq_rope((q, k), self.cos, self.sin, positions, self.head_dim, out=(q, k))
        return q, k, v

    def _slots(self, seq, positions):
        """Where the tokens at `positions` of sequences `seq` go."""
        page = self.table[seq, (positions // self.page_size).long()]
        return page * self.page_size + (positions % self.page_size).to(torch.int32)

    def prompt(self, seq, x):
        """The tokens x [n][hidden] of sequence `seq`, which is empty so far, into the cache -> the block's attention
        output [n][hidden].  Every token is a sequence of its own to the attention call, one longer than the one
        before, over the same pages."""
        n = x.shape[0]
        positions = torch.arange(n, dtype=torch.int32, device="cuda")
        q, k, v = self._qkv(x, positions)
        dq.wq_kv_write(self.cache, k, v, self._slots(seq, positions).contiguous())
        self.lens[seq] = n
        self.longest = max(self.longest, n)
        pages = self.table[seq, : -(-n // self.page_size)]
        y = dq.wq_attn_decode(self.cache, q, pages.repeat(n, 1), positions + 1, max_len=n)
        return dq.wq_linear(self.weights["o"], y)

    def step(self, x):
        """One new token per sequence, x [seqs][hidden] -> the block's attention output [seqs][hidden]."""
        positions = self.lens.clone()
        q, k, v = self._qkv(x, positions)
        slots = self._slots(torch.arange(self.seqs, device="cuda"), positions)
        dq.wq_kv_write(self.cache, k, v, slots)
        self.lens += 1
        self.longest += 1
        y = dq.wq_attn_decode(self.cache, q, self.table, self.lens, max_len=self.longest)
        return dq.wq_linear(self.weights["o"], y)


def main():
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--bits", type=int, default=8, choices=(4, 8, 16))
    ap.add_argument("--seqs", type=int, default=8)
    ap.add_argument("--prompt", type=int, default=500)
    ap.add_argument("--steps", type=int, default=32)
    a = ap.parse_args()
    if min(a.seqs, a.prompt, a.steps) < 1:
        ap.error("--seqs, --prompt and --steps must be positive")
    b = AttentionBlock(a.seqs, a.prompt + a.steps, cache_bits=a.bits)
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    for s in range(a.seqs):
        b.prompt(s, torch.randn((a.prompt, 2560), generator=g, device="cuda").half())
    xs = torch.randn((a.steps, a.seqs, 2560), generator=g, device="cuda").half()
    torch.cuda.synchronize()
    t = time.perf_counter()
    for x in xs:
        y = b.step(x)
    torch.cuda.synchronize()
    dt = (time.perf_counter() - t) / a.steps
    print(f"{a.seqs} sequences of {a.prompt} + {a.steps} tokens, {a.bits}-bit cache: {dt * 1e6:.0f} us a step, "
          f"output rms {y.float().square().mean().sqrt().item():.4f}")


if __name__ == "__main__":
    main()
