"""The host's plans of the attention side's calls: workspace sizes at the
extremes of their arguments, grids too large for a launch, and the planning
itself under AddressSanitizer and UndefinedBehaviorSanitizer
(``tests/host/kv_plan_check.cpp``).  CPU only; pointers are never
dereferenced."""

import ctypes
import os
import subprocess

import pytest

import dequant_gemv_rht_amd as dq
import large_cases as LC

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
P = 1 << 20          # an aligned address that is never touched
ENDS = (0, 1, 14, 15, 16)


def cache(bits=8, head_dim=128, kv_heads=8, page_size=64):
    return ctypes.byref(dq.WqKvCache(bits, head_dim, kv_heads, page_size, 10000, P, P, P, P, None, 0))


@pytest.mark.parametrize("bits,head_dim", [(4, 64), (8, 128), (16, 256)])
@pytest.mark.parametrize("seqs,max_len", [(1, 129), (1, 32001), (3, 5000), (64, 16381), (1, 2 ** 31 - 16385)])
def test_a_window_past_the_lengths_hides_nothing(bits, head_dim, seqs, max_len):
    size = lambda w: dq.lib().wq_attn_decode_workspace(cache(bits, head_dim), seqs, 32, max_len, w)   # noqa: E731
    full = size(0)
    assert 0 < full < 2 ** 63
    for w in {max_len + e for e in ENDS} | {2 ** b - 1 - e for b in (32, 62, 63) for e in ENDS}:
        assert size(w) == full, w
    # and a call with such a window needs that workspace
    need = ctypes.c_size_t(full)
    table = -(-max_len // 64)
    for w in (max_len, 2 ** 63 - 16, 2 ** 63 - 15, 2 ** 63 - 1):
        a = (cache(bits, head_dim), P, 32 * head_dim, 32, seqs, P, table, P, max_len, w, 1.0, P, 32 * head_dim)
        assert dq.lib().wq_attn_decode(*a, None, need, None) == dq.WQ_E_WORKSPACE
        assert dq.lib().wq_attn_decode(*a, P, full - 1, None) == dq.WQ_E_WORKSPACE


def test_a_wider_window_never_needs_less():
    for seqs in (1, 3, 64):
        sizes = [dq.lib().wq_attn_decode_workspace(cache(), seqs, 32, 32001, w)
                 for w in (1, 15, 16, 17, 128, 129, 1000, 5105, 5106, 20000, 31985, 31986, 31987, 32000, 32001, 2 ** 63 - 1)]
        assert sizes == sorted(sizes)


@pytest.fixture(scope="module")
def planner(tmp_path_factory):
    exe = str(tmp_path_factory.mktemp("plan") / "plan")
    csrc = os.path.join(ROOT, "dequant_gemv_rht_amd", "csrc", "kv_plan.cpp")
    r = subprocess.run(["g++", "-std=c++17", "-g", "-O1", "-fsanitize=address,undefined", "-fno-sanitize-recover=all",
                        "-D__HIP_PLATFORM_AMD__", "-isystem", "/opt/rocm/include", csrc,
                        os.path.join(ROOT, "tests", "host", "kv_plan_check.cpp"), "-o", exe], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-2000:]
    return exe


def test_plans_under_asan_ubsan(planner):
    r = subprocess.run([planner], capture_output=True, text=True, timeout=300,
                       env=dict(os.environ, ASAN_OPTIONS="detect_leaks=0", UBSAN_OPTIONS="print_stacktrace=1"))
    assert r.returncode == 0 and "checked" in r.stdout, r.stdout[-500:] + r.stderr[-2000:]


def test_too_many_workgroups_are_refused_on_the_host():
    lib, d = dq.lib(), 256
    # the joining kernel's workgroups are too many, the split kernel's are not
    seqs, group, max_len = (1 << 20) + 5, 16, 9 * 5120
    a = (cache(8, d, 1), P, group * d, group, seqs, P, -(-max_len // 64), P, max_len, 0, 1.0, P, group * d, P, 2 ** 63, None)
    assert lib.wq_attn_decode(*a) == dq.WQ_E_UNSUPPORTED, lib.wq_last_error()
    assert "workgroups" in lib.wq_last_error().decode()
    # the split kernel's
    seqs, group, max_len = 1 << 24, 2, 5120
    a = (cache(8, d, 1), P, group * d, group, seqs, P, -(-max_len // 64), P, max_len, 0, 1.0, P, group * d, P, 2 ** 63, None)
    assert lib.wq_attn_decode(*a) == dq.WQ_E_UNSUPPORTED, lib.wq_last_error()
    # rows of a cache
    tokens = (1 << 28) + 100
    assert lib.wq_kv_write(cache(8, d, 1), P, d, P, d, P, tokens, None) == dq.WQ_E_UNSUPPORTED, lib.wq_last_error()
    assert lib.wq_kv_read(cache(8, d, 1), P, tokens, P, d, P, d, None) == dq.WQ_E_UNSUPPORTED, lib.wq_last_error()
    assert "too many for one launch" in lib.wq_last_error().decode()


def plans(planner, lines):
    r = subprocess.run([planner, "-"], input="\n".join(lines) + "\n", capture_output=True, text=True, timeout=60)
    assert r.returncode == 0, r.stderr
    return [tuple(map(int, line.split())) for line in r.stdout.splitlines()]


def test_large_cases_enter_the_large_forms(planner):
    ask = lambda cases: plans(planner, [f"attn {c.bits} {c.d} {c.seqs} {c.heads} {c.group} {c.max_len} {c.window}"   # noqa: E731
                                        for c in cases])
    for c, (splits, run, _) in zip(LC.STEPS, ask(LC.STEPS)):
        assert splits == 1 and run >= 4 * 128, c
    for c, (splits, run, _) in zip(LC.MASKED + LC.MOVING, ask(LC.MASKED + LC.MOVING)):
        assert splits == 1 and run >= 3 * 128, c
    for c, (splits, run, _) in zip(LC.UNWRITTEN, ask(LC.UNWRITTEN)):
        assert splits == 64 // c.seqs and run == 2048 // splits, c
    for c, (splits, run, _) in zip(LC.SPLIT_STEPS, ask(LC.SPLIT_STEPS)):
        assert splits > 1 and run >= 4 * 128, c
    for c, (splits, _, waves) in zip(LC.JOINS, ask(LC.JOINS)):
        assert waves == 4 and splits > 4 * (4 * 64 * 8 // c.d), c   # four asked for at once by each of a head's groups of lanes
    for c, (quads, _) in zip(LC.ROWS, plans(planner, [f"rows {c.d} {c.tokens} {c.heads}" for c in LC.ROWS])):
        assert quads == (2 if c.d == 256 else 4), c
    for c, (rounds,) in zip(LC.ROPE, plans(planner, [f"rope {c.tokens} {c.rot} {c.heads}" for c in LC.ROPE])):
        assert rounds == 4, c
    more = [c for c in LC.ROPE if c.heads > 4 * (64 // (c.rot // 16))]
    assert more and len(more) < len(LC.ROPE)
