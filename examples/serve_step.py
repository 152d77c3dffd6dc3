"""Steps of a server with many requests, each with pages, an adapter and sampling settings of its own.

    python examples/serve_step.py [--seqs 8] [--prompt 100] [--steps 32] [--adapters 4]

Embedding, one attention block and the output head, with synthetic weights.
A step takes the new tokens of every request, a whole prompt or one, in rows
side by side:

    pages, slots and positions of the rows           (wq_kv_slots)
    the tokens' rows of the embedding                (wq_embed)
    q, k, v and each request's adapter beside them   (wq_linear_batch, wq_lora)
    rotary positions, the cache, attention           (wq_rope, wq_kv_write, wq_attn_decode)
    the output projection, with adapters             (wq_linear, wq_lora)
    the head over each request's last row            (wq_linear)
    each request's next token                        (wq_sample)
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


class Server:
    """`seqs` places for requests of up to `max_len` tokens, `pages` pages for all of them."""

    def __init__(self, seqs, max_len, pages, vocab=8192, hidden=512, q_heads=8, kv_heads=2, head_dim=64, page_size=16,
                 cache_bits=16, adapters=4, rank=16, base=1e4, seed=0):
        rng = np.random.default_rng(seed)
        self.head_dim, self.page_size, self.pages, self.hidden = head_dim, page_size, pages, hidden
        words = lambda k: torch.from_numpy(W.sign_bits(k, rng).view(np.int32)).cuda()  # noqa: E731
        weight = lambda k, n: torch.from_numpy(W.weight(k, n, rng)).cuda()  # noqa: E731
        table = weight(hidden, vocab)
        self.table = dq.quantize_weight(table, 8)             # embedding and head
        shapes = {"q": (hidden, q_heads * head_dim), "k": (hidden, kv_heads * head_dim), "v": (hidden, kv_heads * head_dim),
                  "o": (q_heads * head_dim, hidden)}
        signs = words(hidden)
        self.weights, self.a, self.b = {}, {}, {}
        for name, (k, n) in shapes.items():
            self.weights[name] = dq.quantize_weight(weight(k, n), 4, words(k) if name == "o" else signs)
            self.a[name] = torch.from_numpy((rng.standard_normal((adapters, rank, k)) * k ** -0.5).astype(np.float16)).cuda()
            self.b[name] = torch.from_numpy((rng.standard_normal((adapters, n, rank)) * 0.05).astype(np.float16)).cuda()
        self.scales = torch.from_numpy(rng.uniform(0.5, 2.0, adapters).astype(np.float32)).cuda()
        self.cache = dq.KVCache.new(pages, page_size, kv_heads, head_dim, cache_bits)
        angle = (torch.arange(max_len, device="cuda", dtype=torch.float64)[:, None]
                 * base ** (-torch.arange(0, head_dim, 2, device="cuda", dtype=torch.float64) / head_dim))
        self.cos, self.sin = angle.cos().float(), angle.sin().float()
        i32 = dict(dtype=torch.int32, device="cuda")
        self.pages_of = torch.full((seqs, -(-max_len // page_size)), -1, **i32)
        self.free, self.used = torch.arange(pages, **i32), torch.zeros(1, **i32)
        self.lens = torch.zeros(seqs, **i32)
        self.adapter = torch.full((seqs,), -1, **i32)          # of each request; -1: none
        # what each request asks for; greedy until told
        f32 = dict(dtype=torch.float32, device="cuda")
        self.settings = {"temperature": torch.zeros(seqs, **f32), "top_k": torch.zeros(seqs, **i32),
                         "top_p": torch.ones(seqs, **f32), "min_p": torch.zeros(seqs, **f32)}

    def step(self, tokens, new_tokens, u):
        """tokens int32 [rows] (the sequences' new tokens one after another, then padding), new_tokens int32 [seqs],
        u fp32 [seqs] -> what the step computed, by name; "ids" int32 [seqs] is each request's next token, -1 for one
        without new tokens or without pages for them."""
        r = {"rows": tokens.shape[0], "lens_before": self.lens, "used_before": self.used}
        r["slots"], r["positions"], r["seq_of"], self.lens, r["last"], self.used = dq.wq_kv_slots(
            self.page_size, self.pages, self.pages_of, self.lens, new_tokens, self.free, self.used, tokens.shape[0])
        row = r["seq_of"].clamp(min=0).long()
        r["adapters"] = torch.where(r["seq_of"] >= 0, self.adapter[row], r["seq_of"])
        r["x"] = dq.wq_embed(self.table, tokens)
        names = ("q", "k", "v")
        r["qkv"] = dq.wq_linear_batch([self.weights[n] for n in names], [r["x"]] * 3)
        q, k, v = r["qkv_adapted"] = dq.wq_lora([self.a[n] for n in names], [self.b[n] for n in names], [r["x"]] * 3,
                                                r["adapters"], r["qkv"], scales=self.scales)
        q, k = r["rotated"] = dq.wq_rope((q, k), self.cos, self.sin, r["positions"], self.head_dim)
        dq.wq_kv_write(self.cache, k, v, r["slots"])
        # every row is a sequence of its own, up to its position; padding has none
        y = r["attention"] = dq.wq_attn_decode(self.cache, q, self.pages_of[row], r["positions"] + 1)
        r["o"] = dq.wq_linear(self.weights["o"], y)
        (h,) = r["o_adapted"] = dq.wq_lora([self.a["o"]], [self.b["o"]], [y], r["adapters"], [r["o"]], scales=self.scales)
        h = r["h"] = (r["x"] + h)[r["last"].clamp(min=0).long()]
        r["logits"] = dq.wq_linear(self.table, h, out_dtype=torch.float32, fuse_rht=False)
        ids, r["logprobs"] = dq.wq_sample(r["logits"], u, **self.settings)
        r["ids"] = torch.where(r["last"] >= 0, ids, r["last"])
        return r


def main():
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--seqs", type=int, default=8)
    ap.add_argument("--prompt", type=int, default=100)
    ap.add_argument("--steps", type=int, default=32)
    ap.add_argument("--adapters", type=int, default=4)
    a = ap.parse_args()
    if min(a.seqs, a.prompt, a.steps, a.adapters) < 1:
        ap.error("--seqs, --prompt, --steps and --adapters must be positive")
    length = a.prompt + a.steps
    s = Server(a.seqs, length, a.seqs * -(-length // 16), adapters=a.adapters)
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    s.adapter.copy_(torch.arange(a.seqs, device="cuda") % (a.adapters + 1) - 1)
    s.settings["temperature"].fill_(0.8)
    s.settings["top_p"].fill_(0.95)
    tokens = torch.randint(0, 8192, (a.seqs * a.prompt,), generator=g, device="cuda").to(torch.int32)
    one = torch.ones(a.seqs, dtype=torch.int32, device="cuda")
    u = torch.rand((a.steps + 1, a.seqs), generator=g, device="cuda")
    ids = s.step(tokens, one * a.prompt, u[0])["ids"]
    torch.cuda.synchronize()
    t = time.perf_counter()
    for i in range(a.steps):
        ids = s.step(ids, one, u[i + 1])["ids"]
    torch.cuda.synchronize()
    dt = (time.perf_counter() - t) / a.steps
    print(f"{a.seqs} requests of {a.prompt} + {a.steps} tokens: {dt * 1e6:.0f} us a step, last tokens {ids.tolist()}")


if __name__ == "__main__":
    main()
