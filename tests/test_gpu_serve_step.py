"""Slots, adapters and sampling in the steps of a server (examples/serve_step.py):
prompts of several lengths and single tokens in one step, padding, a request
that finds no pages, adapters and settings of each request.  Every call is
checked against the oracle on the inputs that the calls before it left, and
the cache holds what was written."""

import os
import sys

import numpy as np
import pytest
import torch

import dequant_gemv_rht_amd as dq
from oracle import serving as O

from gpu_util import say
from test_gpu_lora import check as check_lora

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

pytestmark = pytest.mark.gpu


def host(t):
    return t.cpu().numpy()


def check_step(s, r, table_before, new, u, settings):
    want = O.kv_slots(s.page_size, s.pages, table_before, host(r["lens_before"]), new, host(s.free), int(r["used_before"].item()),
                      r["rows"])
    got = (r["slots"], r["positions"], r["seq_of"], s.lens, r["last"], s.used, s.pages_of)
    for g, w in zip(got, want):
        assert np.array_equal(host(g), w)
    adapters = host(r["adapters"])
    for names, x, bases, ys in ((("q", "k", "v"), r["x"], r["qkv"], r["qkv_adapted"]),
                                (("o",), r["attention"], [r["o"]], r["o_adapted"])):
        for name, base, y in zip(names, bases, ys):
            w, off = O.lora(host(s.a[name]), host(s.b[name]), host(x), adapters, host(base), host(s.scales))
            check_lora(y, w, off, False, name)
    # what the step wrote is in the cache (fp16: as it was)
    k, v = dq.wq_kv_read(s.cache, r["slots"])
    live = host(r["slots"]) >= 0
    assert np.array_equal(host(k)[live], host(r["rotated"][1])[live]) and np.array_equal(host(v)[live], host(r["qkv_adapted"][2])[live])
    assert (host(r["attention"])[~live] == 0).all()
    # one token's attention sees it and those before it: a sequence's first token gets its own value
    first = np.flatnonzero(host(r["positions"]) == 0)
    for i in first:
        value = np.repeat(host(r["qkv_adapted"][2])[i].reshape(-1, s.head_dim), host(r["attention"]).shape[1] // v.shape[1], axis=0)
        assert np.abs(host(r["attention"])[i] - value.reshape(-1)).max() <= 2.0 ** -10 * np.abs(value).max()
    logits, ids = host(r["logits"]), host(r["ids"])
    for i in range(len(ids)):
        if host(r["last"])[i] < 0:
            assert ids[i] == -1
            continue
        token, chance = O.sample(logits[i], u[i], **{n: v[i] for n, v in settings.items()})
        assert ids[i] == token
        assert abs(host(r["logprobs"])[i] - chance) <= abs(chance) * 2.0 ** -23 + 1e-9


def test_steps_of_a_server():
    import serve_step

    seqs = 6
    s = serve_step.Server(seqs, 128, 15, adapters=3)
    rng = np.random.default_rng(5)
    s.adapter.copy_(torch.tensor([0, 2, -1, 2, 1, 0], dtype=torch.int32))
    settings = {"temperature": np.array([0.0, 0.7, 1.0, 1.3, 0.9, 0.6], np.float32), "top_k": np.array([0, 40, 0, 5, 0, 100]),
                "top_p": np.array([1.0, 0.9, 1.0, 1.0, 0.8, 0.95], np.float32), "min_p": np.array([0, 0, 0.05, 0, 0, 0.02], np.float32)}
    for n, v in settings.items():
        s.settings[n].copy_(torch.from_numpy(v.astype(np.int32 if n == "top_k" else np.float32)))
    # three prompts; then more prompts among single tokens; then a step that runs out of pages; then tokens alone
    plan = [[17, 40, 0, 16, 0, 0], [1, 1, 33, 1, 0, 0], [1, 1, 1, 1, 90, 1], [1, 1, 1, 0, 64, 1], [1, 1, 1, 1, 1, 1], [1, 0, 1, 1, 1, 1]]
    ids = np.full(seqs, -1)
    served = []
    for turn, new in enumerate(plan):
        say("server step", turn, new)
        rows = []
        for i, n in enumerate(new):
            rows += [ids[i]] if n == 1 and ids[i] >= 0 else rng.integers(0, 8192, n).tolist()
        rows += [0] * 5                                       # padding
        u = rng.random(seqs).astype(np.float32)
        before = host(s.pages_of).copy()
        r = s.step(torch.tensor(rows, dtype=torch.int32, device="cuda"), torch.tensor(new, dtype=torch.int32, device="cuda"),
                   torch.from_numpy(u).cuda())
        check_step(s, r, before, new, u, settings)
        got = host(r["ids"])
        ids = np.where(got >= 0, got, ids)
        served.append((host(r["last"]) >= 0).tolist())
    assert served[2][4] is False and served[3][4] is True     # 90 tokens found no pages, 64 did
    assert all(served[0][i] for i in (0, 1, 3))


def test_captured_step():
    """A decode step as a graph: the same tokens as step by step."""
    import serve_step

    seqs, steps = 4, 6
    tokens = torch.arange(40, dtype=torch.int32, device="cuda") * 7
    new = torch.tensor([10, 5, 20, 5], dtype=torch.int32, device="cuda")
    one = torch.ones(seqs, dtype=torch.int32, device="cuda")
    u = torch.rand((steps, seqs), generator=torch.Generator().manual_seed(3)).cuda()
    runs = []
    for captured in (False, True):
        s = serve_step.Server(seqs, 64, 16, adapters=2)
        s.adapter.copy_(torch.tensor([1, -1, 0, 1], dtype=torch.int32))
        s.settings["temperature"].fill_(0.9)
        s.settings["top_p"].fill_(0.9)
        ids = s.step(tokens, new, u[0])["ids"]
        lens, used, table = s.lens.clone(), s.used.clone(), s.pages_of.clone()
        out = []
        if captured:
            held, now, lens_in, used_in = ids.clone(), u[0].clone(), s.lens, s.used
            side = torch.cuda.Stream()
            side.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(side):   # a step outside, taken back
                s.step(held, one, now)
            torch.cuda.current_stream().wait_stream(side)
            s.lens, s.used = lens_in, used_in
            s.pages_of.copy_(table)
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g):
                r = s.step(held, one, now)
                held.copy_(r["ids"])
                lens_in.copy_(s.lens)
                used_in.copy_(s.used)
            lens_in.copy_(lens)
            used_in.copy_(used)
            s.pages_of.copy_(table)
            held.copy_(ids)
        for i in range(1, steps):
            if captured:
                now.copy_(u[i])
                g.replay()
                torch.cuda.synchronize()
                torch.randn(50, device="cuda").sum().item()   # eager work between replays
                out.append(held.tolist())
            else:
                ids = s.step(ids, one, u[i])["ids"]
                out.append(ids.tolist())
        runs.append(out)
    assert runs[0] == runs[1]


def test_two_streams_at_once():
    """Calls on two streams, each with a workspace of its own, while the other's run."""
    g = torch.Generator(device="cuda")
    g.manual_seed(2)
    x = [torch.randn((40, 50000), generator=g, device="cuda") * 3 for _ in range(2)]
    u = [torch.rand(40, generator=g, device="cuda") for _ in range(2)]
    p = torch.full((40,), 0.9, device="cuda")
    a, b = (torch.randn(s, generator=g, device="cuda").half() for s in ((5, 16, 2560), (5, 4096, 16)))
    rows = [torch.randn((64, 2560), generator=g, device="cuda").half() for _ in range(2)]
    base = torch.randn((64, 4096), generator=g, device="cuda").half()
    ids = [torch.randint(-1, 5, (64,), generator=g, device="cuda").to(torch.int32) for _ in range(2)]
    both = lambda i: (*dq.wq_sample(x[i], u[i], top_p=p), *dq.wq_lora([a], [b], [rows[i]], ids[i], [base]))  # noqa: E731
    want = [[t.clone() for t in both(i)] for i in range(2)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [[], []]
    for turn in range(10):
        for i, st in enumerate(streams):
            with torch.cuda.stream(st):
                got[i].append(both(i))
    torch.cuda.synchronize()
    for i in range(2):
        for out in got[i]:
            assert all(torch.equal(o, w) for o, w in zip(out, want[i]))


def test_the_example_runs(capsys, monkeypatch):
    import serve_step

    monkeypatch.setattr(sys, "argv", ["serve_step.py", "--seqs", "3", "--prompt", "20", "--steps", "4", "--adapters", "2"])
    serve_step.main()
    assert "us a step" in capsys.readouterr().out
