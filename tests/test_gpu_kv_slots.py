"""wq_kv_slots against the oracle, number for number: no sequences, no rows,
sequences without new tokens, pages that run out, tables and steps that are
too small, lists past their end, padded table rows, several workgroups and
turns."""

import numpy as np
import pytest
import torch

import dequant_gemv_rht_amd as dq
from oracle import serving as O

from gpu_util import say

pytestmark = pytest.mark.gpu


def gpu(x):
    return torch.tensor(np.asarray(x, dtype=np.int32), device="cuda")


def check(page, pages, table, lens, new, free, used, tokens, ld=None):
    table = np.asarray(table, np.int32)
    want = O.kv_slots(page, pages, table, lens, new, free, used, tokens)
    ld = ld or table.shape[1]
    wide = torch.full((len(lens), ld), -7, dtype=torch.int32, device="cuda")
    wide[:, : table.shape[1]] = gpu(table)
    view = wide[:, : table.shape[1]]
    args = (page, pages, view, gpu(lens), gpu(new), gpu(free), gpu([used]), tokens)
    for _ in range(2):   # the second call finds the table as the first left it
        got = dq.wq_kv_slots(*args)
        torch.cuda.synchronize()
        for name, g, w in zip(("slots", "positions", "seq_of", "lens", "last", "used", "table"), (*got, view), want):
            assert g.dtype == torch.int32 and np.array_equal(g.cpu().numpy(), w), name
    assert (wide[:, table.shape[1]:] == -7).all()
    return got


def random_case(rng, seqs, page, held, most, empty=0.2):
    lens = rng.integers(0, held + 1, seqs)
    new = np.where(rng.random(seqs) < empty, 0, rng.integers(0, most + 1, seqs))
    cols = (held + most) // page + 2
    order = rng.permutation(seqs * cols + 50)
    table = order[: seqs * cols].reshape(seqs, cols)
    free = rng.permutation(seqs * cols + 50)[: int((-(-(lens + new) // page) + lens * 0).sum()) + 5]
    return table, lens, new, free, seqs * cols + 50


@pytest.mark.parametrize("seqs,page,held,most", [(1, 16, 0, 1), (1, 64, 100, 1), (3, 16, 40, 33), (64, 16, 500, 1),
                                                 (255, 32, 70, 4), (1023, 16, 50, 3), (1024, 16, 50, 3), (1025, 16, 50, 3),
                                                 (2500, 128, 300, 2), (9, 64, 0, 2047), (5, 16, 3000, 1500)])
def test_against_oracle(seqs, page, held, most):
    rng = np.random.default_rng(seqs)
    table, lens, new, free, pages = random_case(rng, seqs, page, held, most)
    total = int(new.sum())
    for used, tokens in ((0, total), (3, total + 77), (2, max(0, total - 5)), (0, 0)):
        say("slots", seqs, page, held, most, used, tokens)
        check(page, pages, table, lens, new, free, used, tokens, ld=table.shape[1] + 3)


@pytest.mark.parametrize("left", [0, 1, 7, 40])
def test_pages_run_out(left):
    rng = np.random.default_rng(left)
    table, lens, new, free, pages = random_case(rng, 60, 16, 90, 40)
    check(16, pages, table, lens, new, free[: left + 4], 4, int(new.sum()))


def test_pages_not_given_out_stay_in_the_list():
    """One page left: the first needs two, the second none and the third one; used counts what was given out."""
    check(16, 8, [[0, -1, -1], [1, -1, -1], [2, -1, -1]], [16, 3, 16], [17, 1, 1], [5], 0, 19)
    check(16, 8, [[1, -1, -1], [2, -1, -1], [0, -1, -1]], [3, 16, 16], [1, 1, 17], [5], 0, 19)


@pytest.mark.parametrize("used", [-1, -2 ** 31, 11, 2 ** 31 - 1])
def test_used_outside_the_list(used):
    check(16, 50, [[1, 2], [3, 4]], [16, 5], [1, 2], list(range(10, 20)), used, 3)


def test_bad_lengths_and_pages():
    say("slots: negative lengths, pages outside the cache, rows that do not fit")
    check(16, 50, [[1, 2], [50, 4], [-3, 9], [7, 8]], [-5, 3, 2, 20], [3, 2, 1, -4], [50, 6, 7], 0, 9)
    check(16, 50, [[1, 2], [3, 4]], [2 ** 31 - 1, 31], [1, 2], [5, 6], 0, 9)
    check(16, 50, [[1, 2], [3, 4]], [0, 0], [2 ** 31 - 1, 2 ** 31 - 1], [5, 6], 0, 9)
    check(16, 50, [[1], [3]], [0, 0], [17, 16], [5, 6], 0, 40)


def test_no_sequences():
    got = check(16, 50, np.zeros((0, 3)), [], [], [1], 0, 5)
    assert got[0].tolist() == [-1] * 5


def test_many_sequences_of_none_then_one():
    seqs = 5000
    new = np.zeros(seqs, np.int64)
    new[-1] = 2100
    check(16, 9000, np.zeros((seqs, 140)), np.zeros(seqs, np.int64), new, np.arange(200), 0, 2100)


def test_given_outputs_are_written_whole_and_alone():
    rng = np.random.default_rng(3)
    table, lens, new, free, pages = random_case(rng, 20, 16, 60, 9)
    tokens = int(new.sum()) + 4
    want = O.kv_slots(16, pages, table, lens, new, free, 0, tokens)
    sizes = [tokens] * 3 + [20, 20, 1]
    bufs = [torch.full((n + 8,), 99, dtype=torch.int32, device="cuda") for n in sizes]
    out = [b[4:4 + n] for b, n in zip(bufs, sizes)]
    got = dq.wq_kv_slots(16, pages, gpu(table), gpu(lens), gpu(new), gpu(free), gpu([0]), tokens, out=out)
    for g, o, b, w in zip(got, out, bufs, want):
        assert g.data_ptr() == o.data_ptr() and np.array_equal(o.cpu().numpy(), w)
        assert (b[:4] == 99).all() and (b[-4:] == 99).all()


def test_captured_steps_advance():
    """A captured step whose lengths and place in the list feed back: every replay against the oracle."""
    seqs, page, tokens = 6, 16, 16
    lens, new = np.array([0, 15, 16, 3, 40, 9]), np.array([1, 1, 2, 0, 1, 3])
    table = np.full((seqs, 8), -1)
    for s in range(seqs):
        for j in range(-(-lens[s] // page)):
            table[s, j] = 10 * s + j
    free = np.arange(70, 99)
    d = {"table": gpu(table), "lens": gpu(lens), "new": gpu(new), "free": gpu(free), "used": gpu([0])}
    out = [torch.zeros(n, dtype=torch.int32, device="cuda") for n in (tokens, tokens, tokens, seqs, seqs, 1)]

    def step():
        dq.wq_kv_slots(page, 120, d["table"], d["lens"], d["new"], d["free"], d["used"], tokens, out=out)
        d["lens"].copy_(out[3])
        d["used"].copy_(out[5])

    stream = torch.cuda.Stream()
    with torch.cuda.stream(stream):
        step()
    torch.cuda.synchronize()
    for name, x in (("table", table), ("lens", lens), ("used", [0])):
        d[name].copy_(gpu(x))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    used = 0
    for turn in range(20):
        g.replay()
        torch.cuda.synchronize()
        want = O.kv_slots(page, 120, table, lens, new, free, used, tokens)
        for o, w in zip((*out, d["table"]), want):
            assert np.array_equal(o.cpu().numpy(), w), turn
        lens, used, table = want[3], int(want[5][0]), want[6]
        torch.randn(100, device="cuda").sum().item()   # eager work between replays
