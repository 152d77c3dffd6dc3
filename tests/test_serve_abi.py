"""Argument checks of the slots, adapters and sampling calls: every defect is
refused on the host, before any HIP call, with a message (CPU only; device
pointers here are never dereferenced)."""

import ctypes

import pytest
import torch

import dequant_gemv_rht_amd as dq

A, U, L, W = dq.WQ_E_ARG, dq.WQ_E_UNSUPPORTED, dq.WQ_E_ALIGN, dq.WQ_E_WORKSPACE
MB = 1 << 20
BIG = 1 << 62


def P(i):
    """An aligned address, a mebibyte to each."""
    return (i + 1) * MB


@pytest.fixture(scope="module")
def lib():
    return dq.lib()


def said(lib, st, status, text):
    assert st == status, lib.wq_last_error()
    assert text in lib.wq_last_error().decode()


# ---------------------------------------------------------------- slots

NAMES = ("page_size", "pages", "table", "ld_table", "table_pages", "lens", "new", "seqs", "free", "free_count", "used",
         "tokens", "slots", "positions", "seq_of", "lens_out", "last", "used_out")
GOOD = (16, 100, P(0), 8, 8, P(1), P(2), 4, P(3), 50, P(4), 64, P(5), P(6), P(7), P(8), P(9), P(10))


@pytest.mark.parametrize("kw,status,text", [
    (dict(page_size=8), U, "page_size=8"), (dict(page_size=24), U, "page_size=24"), (dict(page_size=-(1 << 31)), U, "page_size"),
    (dict(page_size=0), U, "page_size"), (dict(pages=0), A, "pages=0"), (dict(pages=1 << 40), U, "2^31"),
    (dict(seqs=-1), A, "seqs=-1"), (dict(tokens=-1), A, "tokens=-1"), (dict(free_count=-1), A, "free_count=-1"),
    (dict(table_pages=-1), A, "table_pages=-1"), (dict(seqs=(1 << 20) + 1), U, "seqs above"),
    (dict(tokens=(1 << 30) + 1), U, "tokens above"), (dict(free_count=1 << 31), U, "free_count"),
    (dict(ld_table=7), A, "ld_table=7"), (dict(ld_table=BIG), U, "address range"), (dict(table=None), A, "non-NULL"),
    (dict(lens=None), A, "non-NULL"), (dict(new=None), A, "non-NULL"), (dict(free=None), A, "non-NULL"),
    (dict(used=None), A, "non-NULL"), (dict(slots=None), A, "non-NULL"), (dict(positions=None), A, "non-NULL"),
    (dict(seq_of=None), A, "non-NULL"), (dict(lens_out=None), A, "non-NULL"), (dict(last=None), A, "non-NULL"),
    (dict(used_out=None), A, "non-NULL"), (dict(lens=P(1) + 2), L, "aligned"), (dict(last=P(9) + 1), L, "aligned"),
    (dict(lens_out=P(1)), A, "overlaps an input"), (dict(used_out=P(4)), A, "overlaps an input"),
    (dict(lens_out=P(2) + 12), A, "overlaps an input"), (dict(slots=P(3) - 252), A, "overlaps an input"),
    (dict(slots=P(6) + 252), A, "outputs overlap"), (dict(table=P(5) - 124), A, "outputs overlap"),
])
def test_bad_slots(lib, kw, status, text):
    args = dict(zip(NAMES, GOOD))
    assert set(kw) <= set(args)
    args.update(kw)
    said(lib, lib.wq_kv_slots(*args.values(), None), status, text)


# ---------------------------------------------------------------- adapters

def adapters(linears=1, **kw):
    base = dict(n=64, k=128, count=4, rank=16, a=P(0), b=P(1), scales=P(2))
    base.update(kw)
    return (dq.WqAdapters * max(linears, 1))(*[dq.WqAdapters(**base) for _ in range(max(linears, 1))])


def lora(lib, count=1, w=None, m=4, ids=P(3), ws=P(30), ws_bytes=1 << 30, null=None, **kw):
    w = adapters(count) if w is None else w
    one = dict(x=P(4), ldx=128, base=P(5), ldb=64, y=P(6), ldy=64, dtype=1)
    one.update(kw)
    vp, i64, i32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32
    n = max(count, 1)
    arr = {k: (vp if k in "x base y".split() else i32 if k == "dtype" else i64) for k in one}
    arr = {k: (t * n)(*[one[k] if not isinstance(one[k], list) else one[k][i] for i in range(n)]) for k, t in arr.items()}
    if null:
        arr[null] = None
    return lib.wq_lora(count, w, arr["x"], arr["ldx"], m, ids, arr["base"], arr["ldb"], arr["y"], arr["ldy"], arr["dtype"],
                       ws, ws_bytes, None)


BAD_ADAPTERS = [
    (dict(rank=0), U, "rank"), (dict(rank=12), U, "rank[0]=12"), (dict(rank=136), U, "rank"), (dict(rank=-8), U, "rank"),
    (dict(n=0), A, "n=0"), (dict(k=0), A, "k=0"), (dict(count=0), A, "count=0"), (dict(count=-1), A, "count=-1"),
    (dict(k=192), A, "multiple of 128"), (dict(n=1 << 30), U, "2^30"), (dict(k=1 << 27), U, "2^27"),
]


@pytest.mark.parametrize("kw,status,text", BAD_ADAPTERS)
def test_bad_adapters(lib, kw, status, text):
    said(lib, lora(lib, w=adapters(**kw)), status, text)
    assert lib.wq_lora_workspace(1, adapters(**kw), 4) == ctypes.c_size_t(-1).value
    assert text in lib.wq_last_error().decode()


@pytest.mark.parametrize("kw,status,text", [
    (dict(count=0), A, "count=0"), (dict(count=9), A, "count=9"), (dict(m=-1), A, "m=-1"), (dict(m=1 << 24), U, "2^24"),
    (dict(ids=None), A, "ids"), (dict(ids=P(3) + 2), L, "ids"), (dict(null="x"), A, "NULL argument"),
    (dict(null="ldb"), A, "NULL argument"), (dict(null="y"), A, "NULL argument"), (dict(null="dtype"), A, "NULL argument"),
    (dict(x=None), A, "non-NULL"), (dict(base=None), A, "non-NULL"), (dict(y=None), A, "non-NULL"),
    (dict(w=adapters(a=None)), A, "non-NULL"), (dict(w=adapters(b=None)), A, "non-NULL"), (dict(dtype=0), A, "dtype"),
    (dict(ldx=120), A, "ldx=120"), (dict(ldb=63), A, "ldb=63"), (dict(ldy=63), A, "ldy=63"), (dict(ldx=132), L, "ldx"),
    (dict(ldx=BIG), U, "address range"), (dict(ldy=BIG), U, "address range"), (dict(x=P(4) + 8), L, "aligned"),
    (dict(base=P(5) + 2), L, "aligned"), (dict(y=P(6) + 2), L, "aligned"), (dict(w=adapters(scales=P(2) + 2)), L, "aligned"),
    (dict(w=adapters(a=P(0) + 8)), L, "aligned"), (dict(y=P(4)), A, "overlaps an input"), (dict(y=P(3)), A, "overlaps an input"),
    (dict(y=P(5) + 16), A, "overlaps an input"), (dict(y=P(5), ldy=72), A, "overlaps an input"),
    (dict(y=P(2)), A, "overlaps an input"), (dict(count=2, y=[P(6), P(6)]), A, "overlap"),
    (dict(count=2, y=[P(5), P(6)]), A, "overlaps an input"),   # in place, and the other linear's base too
    (dict(ws=None), W, "workspace"), (dict(ws_bytes=255), W, "workspace"), (dict(ws=P(30) + 8), L, "workspace"),
])
def test_bad_lora(lib, kw, status, text):
    said(lib, lora(lib, **kw), status, text)


@pytest.mark.parametrize("kw,status,text", [
    (dict(y=P(0)), A, "overlaps an input"), (dict(y=P(1) + 16), A, "overlaps an input"),      # a, b
    (dict(ws=P(6)), A, "workspace overlaps y[0]"), (dict(ws=P(5) + 16), A, "workspace overlaps an input"),
    (dict(ws=P(0)), A, "workspace overlaps an input"), (dict(ws=P(3)), A, "workspace overlaps an input"),
    (dict(w=adapters(count=2 ** 31 - 1, rank=128, k=1 << 26)), U, "address range"),
    # columns of one wide array: a column in common, another row stride, the next row's first column
    (dict(count=2, y=[P(6), P(6) + 112], ldy=128), A, "overlap"), (dict(count=2, y=[P(6), P(6) + 128], ldy=[128, 136]), A, "overlap"),
    (dict(count=2, y=[P(6), P(6) + 144], ldy=128), A, "overlap"), (dict(count=2, y=[P(6) + 144, P(6)], ldy=128), A, "overlap"),
    (dict(count=2, y=[P(6), P(6) + 128], ldy=128, ws=None), W, "workspace"),                  # none: goes on to the next check
    (dict(count=2, y=[P(6) + 256 + 128, P(6)], ldy=128, ws=None), W, "workspace"),
])
def test_lora_arrays_apart(lib, kw, status, text):
    said(lib, lora(lib, **kw), status, text)


def test_lora_workspace(lib):
    assert lib.wq_lora_workspace(1, adapters(), 0) == 0
    sizes = [lib.wq_lora_workspace(1, adapters(), m) for m in (0, 1, 2, 16, 17, 64, 256, 257, 1000, 5000, (1 << 24) - 1)]
    assert sizes == sorted(sizes) and sizes[1] >= 16 * 4
    assert lib.wq_lora_workspace(2, adapters(2), 5) == 2 * lib.wq_lora_workspace(1, adapters(), 5)
    assert lib.wq_lora_workspace(1, None, 5) == ctypes.c_size_t(-1).value
    assert lora(lib, m=0, ids=None, x=None, base=None, y=None, ws=None) == dq.WQ_OK


# ---------------------------------------------------------------- sampling

SAMPLE = dict(logits=P(0), dtype=2, rows=4, vocab=1000, ldl=1000, u=P(1), temperature=P(2), top_k=P(3), top_p=P(4),
              min_p=P(5), ids=P(6), logprobs=P(7), ws=P(8), ws_bytes=1 << 30)


@pytest.mark.parametrize("kw,status,text", [
    (dict(rows=-1), A, "rows=-1"), (dict(vocab=0), A, "vocab=0"), (dict(vocab=-5), A, "vocab=-5"),
    (dict(rows=(1 << 20) + 1), U, "2^20"), (dict(vocab=(1 << 20) + 1, ldl=1 << 21), U, "2^20"), (dict(dtype=0), A, "dtype=0"),
    (dict(dtype=3), A, "dtype=3"), (dict(ldl=999), A, "ldl=999"), (dict(ldl=BIG), U, "address range"),
    (dict(logits=None), A, "non-NULL"), (dict(u=None), A, "non-NULL"), (dict(ids=None), A, "non-NULL"),
    (dict(logits=P(0) + 8), L, "aligned"), (dict(u=P(1) + 2), L, "aligned"), (dict(top_k=P(3) + 1), L, "aligned"),
    (dict(logprobs=P(7) + 2), L, "aligned"), (dict(ids=P(1)), A, "overlaps an input"), (dict(ids=P(0) + 4000), A, "overlaps"),
    (dict(logprobs=P(4) + 12), A, "overlaps an input"), (dict(logprobs=P(6) + 12), A, "outputs overlap"),
])
def test_bad_sample(lib, kw, status, text):
    said(lib, lib.wq_sample(*{**SAMPLE, **kw}.values(), None), status, text)


@pytest.mark.parametrize("ws,text", [(P(0), "an input"), (P(4), "an input"), (P(6), "an output"), (P(7), "an output")])
def test_sample_workspace_apart(lib, ws, text):
    said(lib, lib.wq_sample(*{**SAMPLE, "ws": ws}.values(), None), A, "workspace overlaps " + text)


def test_sample_workspace(lib):
    for rows, vocab in ((-1, 10), (1, 0), ((1 << 20) + 1, 5), (5, (1 << 20) + 1)):
        assert lib.wq_sample_workspace(rows, vocab) == ctypes.c_size_t(-1).value
        assert "wq_sample_workspace" in lib.wq_last_error().decode()
    need = lib.wq_sample_workspace(4, 200000)
    if need:
        args = {**SAMPLE, "vocab": 200000, "ldl": 200000}
        said(lib, lib.wq_sample(*{**args, "ws_bytes": need - 1}.values(), None), W, "workspace")
        said(lib, lib.wq_sample(*{**args, "ws": None}.values(), None), W, "workspace")
        said(lib, lib.wq_sample(*{**args, "ws": P(8) + 8}.values(), None), L, "workspace")
    assert lib.wq_sample(*{**SAMPLE, "rows": 0, "logits": None, "u": None, "ids": None}.values(), None) == dq.WQ_OK


# ---------------------------------------------------------------- the binding

def test_binding_refuses_host_tensors_and_non_tensors():
    i = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError, match="GPU"):
        dq.wq_kv_slots(16, 10, torch.zeros((2, 2), dtype=torch.int32), i, i, i, i[:1], 2)
    with pytest.raises(TypeError, match="lens"):
        dq.wq_kv_slots(16, 10, i, 5, i, i, i, 2)
    h = torch.zeros((1, 8, 128), dtype=torch.float16)
    with pytest.raises(ValueError, match="GPU"):
        dq.wq_lora([h], [h], [h[0]], i, [h[0]])
    with pytest.raises(ValueError, match="linears"):
        dq.wq_lora([], [], [], i, [])
    with pytest.raises(ValueError, match="b: 0 given"):
        dq.wq_lora([h], [], [h[0]], i, [h[0]])
    with pytest.raises(ValueError, match="GPU"):
        dq.wq_sample(torch.zeros((2, 5)), torch.zeros(2))
    with pytest.raises(TypeError, match="logits"):
        dq.wq_sample(None, torch.zeros(2))
    with pytest.raises(dq.WqError):
        dq.wq_sample_workspace(1, 0)
