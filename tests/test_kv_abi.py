"""Argument checks of the key-value cache, attention and rotary calls: every
defect is refused on the host, before any HIP call, with a message (CPU
only; pointers here are never dereferenced, except the host arrays of
wq_rope)."""

import ctypes

import pytest
import torch

import dequant_gemv_rht_amd as dq

P = 1 << 20          # an aligned address that is never touched


@pytest.fixture(scope="module")
def lib():
    return dq.lib()


def cache(**kw):
    base = dict(bits=8, head_dim=128, kv_heads=2, page_size=16, pages=10, k=P, v=P, k_params=P, v_params=P,
                rht_signs=None, rht_block=0)
    base.update(kw)
    return ctypes.byref(dq.WqKvCache(**base))


A, U, L = dq.WQ_E_ARG, dq.WQ_E_UNSUPPORTED, dq.WQ_E_ALIGN

BAD_CACHES = [
    (dict(bits=3), U, "bits=3"), (dict(bits=0), U, "bits=0"), (dict(head_dim=96), U, "head_dim=96"),
    (dict(kv_heads=0), A, "kv_heads=0"), (dict(kv_heads=1 << 30), U, "kv_heads"),
    (dict(page_size=8), U, "page_size=8"), (dict(page_size=48), U, "page_size=48"), (dict(page_size=0), U, "page_size=0"),
    (dict(page_size=-(1 << 31)), U, "page_size"), (dict(pages=0), A, "pages=0"), (dict(pages=1 << 40), U, "2^31"),
    (dict(k=None), A, "non-NULL"), (dict(v=None), A, "non-NULL"), (dict(k=P + 8), L, "aligned"),
    (dict(k_params=None), A, "k_params"), (dict(v_params=None, bits=4), A, "k_params"), (dict(v_params=P + 4), L, "aligned"),
    (dict(rht_signs=P, rht_block=64), U, "rht_block=64"), (dict(rht_signs=P, rht_block=128, head_dim=64), U, "head_dim"),
    (dict(rht_signs=P + 4, rht_block=128), L, "rht_signs"),
]


@pytest.mark.parametrize("kw,status,text", BAD_CACHES)
def test_bad_caches(lib, kw, status, text):
    c = cache(**kw)
    calls = [lambda: lib.wq_kv_write(c, P, 256, P, 256, P, 1, None),
             lambda: lib.wq_kv_read(c, P, 1, P, 256, P, 256, None),
             lambda: lib.wq_attn_decode(c, P, 1024, 8, 1, P, 4, P, 64, 0, 1.0, P, 1024, P, 1 << 40, None)]
    for f in calls:
        assert f() == status
        assert text in lib.wq_last_error().decode()
    assert lib.wq_attn_decode_workspace(c, 1, 8, 64, 0) == ctypes.c_size_t(-1).value
    assert text in lib.wq_last_error().decode()


def test_null_cache(lib):
    assert lib.wq_kv_write(None, P, 256, P, 256, P, 1, None) == A
    assert "NULL" in lib.wq_last_error().decode()


@pytest.mark.parametrize("kw,status,text", [
    (dict(k=None), A, "non-NULL"), (dict(v=None), A, "non-NULL"), (dict(slots=None), A, "non-NULL"),
    (dict(ldk=248), A, "ldk=248"), (dict(ldv=0), A, "ldv=0"), (dict(ldk=260), L, "multiples of 8"),
    (dict(tokens=-1), A, "tokens=-1"), (dict(tokens=1 << 40), U, "tokens"), (dict(k=P + 8), L, "aligned"),
    (dict(slots=P + 2), L, "aligned"), (dict(ldk=(1 << 62), tokens=9), U, "address range"),
])
def test_bad_rows(lib, kw, status, text):
    a = dict(k=P, ldk=256, v=P, ldv=256, slots=P, tokens=1)
    a.update(kw)
    assert lib.wq_kv_write(cache(), a["k"], a["ldk"], a["v"], a["ldv"], a["slots"], a["tokens"], None) == status
    assert text in lib.wq_last_error().decode()
    assert lib.wq_kv_read(cache(), a["slots"], a["tokens"], a["k"], a["ldk"], a["v"], a["ldv"], None) == status
    assert text in lib.wq_last_error().decode()


def test_nothing_to_do(lib):
    assert lib.wq_kv_write(cache(), None, 0, None, 0, None, 0, None) == dq.WQ_OK
    assert lib.wq_kv_read(cache(), None, 0, None, 0, None, 0, None) == dq.WQ_OK
    assert lib.wq_attn_decode(cache(), None, 0, 8, 0, None, 0, None, 0, 0, 1.0, None, 0, None, 0, None) == dq.WQ_OK


@pytest.mark.parametrize("kw,status,text", [
    (dict(q=None), A, "non-NULL"), (dict(table=None), A, "non-NULL"), (dict(lens=None), A, "non-NULL"),
    (dict(out=None), A, "non-NULL"), (dict(q_heads=0), A, "q_heads=0"), (dict(q_heads=3), A, "q_heads=3"),
    (dict(q_heads=-2), A, "q_heads"), (dict(q_heads=1 << 30), U, "q_heads"), (dict(seqs=-1), A, "seqs=-1"),
    (dict(seqs=1 << 40), U, "seqs"), (dict(max_len=-1), A, "max_len=-1"), (dict(window=-1), A, "window=-1"),
    (dict(max_len=2 ** 31 - 16384), U, "max_len"), (dict(max_len=65), A, "ld_table=4"), (dict(ld_table=-1), A, "ld_table"),
    (dict(ldq=1016), A, "ldq=1016"), (dict(ldo=8), A, "ldo=8"), (dict(ldq=1028), L, "multiples of 8"),
    (dict(scale=float("nan")), A, "scale"), (dict(scale=float("inf")), A, "scale"), (dict(q=P + 8), L, "aligned"),
    (dict(out=P + 2), L, "aligned"), (dict(table=P + 2), L, "aligned"), (dict(lens=P + 1), L, "aligned"),
    (dict(ldq=1 << 62, seqs=5), U, "address range"),
])
def test_bad_attention(lib, kw, status, text):
    a = dict(q=P, ldq=1024, q_heads=8, seqs=1, table=P, ld_table=4, lens=P, max_len=64, window=0, scale=1.0, out=P,
             ldo=1024)
    a.update(kw)
    st = lib.wq_attn_decode(cache(), a["q"], a["ldq"], a["q_heads"], a["seqs"], a["table"], a["ld_table"], a["lens"],
                            a["max_len"], a["window"], a["scale"], a["out"], a["ldo"], P, 1 << 40, None)
    assert st == status, lib.wq_last_error()
    assert text in lib.wq_last_error().decode()


def test_attention_workspace_is_checked(lib):
    need = lib.wq_attn_decode_workspace(cache(pages=10000), 4, 8, 100000, 0)
    if need:
        args = (cache(pages=10000), P, 1024, 8, 4, P, 6250, P, 100000, 0, 1.0, P, 1024)
        assert lib.wq_attn_decode(*args, P, need - 1, None) == dq.WQ_E_WORKSPACE
        assert "workspace" in lib.wq_last_error().decode()
        assert lib.wq_attn_decode(*args, None, need, None) == dq.WQ_E_WORKSPACE
        assert lib.wq_attn_decode(*args, P + 8, need, None) == L
    # it never shrinks as the bound of the lengths grows, and a window bounds it
    sizes = [lib.wq_attn_decode_workspace(cache(pages=10000), 4, 8, n, 0) for n in (0, 1, 100, 1000, 10000, 100000)]
    assert sizes == sorted(sizes)
    assert lib.wq_attn_decode_workspace(cache(), 0, 8, 64, 0) == 0
    wide = dq.WqKvCache(8, 64, 1, 16, 10, P, P, P, P, None, 0)   # one head shared by 2^25
    assert lib.wq_attn_decode_workspace(ctypes.byref(wide), 1, 2 ** 25 - 1, 2 ** 31 - 16385, 0) < 2 ** 63
    big = lib.wq_attn_decode_workspace(cache(), 2 ** 31 // 8 - 1, 8, 2 ** 31 - 16385, 0)   # no overflow
    assert 2 ** 31 < big < 2 ** 63


def rope(lib, **kw):
    a = dict(count=1, x=P, ldx=256, y=P, ldy=256, heads=2, tokens=3, d=128, rot=128, cos=P, sin=P, rows=10, pos=P,
             ld_pos=3, axes=2, axis=bytes([0, 1] * 32), flags=0)
    a.update(kw)
    c = max(1, min(a["count"], 9))
    arr = lambda t, v: (t * c)(*[v] * c)   # noqa: E731
    return lib.wq_rope(a["count"], arr(ctypes.c_void_p, a["x"]), arr(ctypes.c_int64, a["ldx"]),
                       arr(ctypes.c_void_p, a["y"]), arr(ctypes.c_int64, a["ldy"]), arr(ctypes.c_int32, a["heads"]),
                       a["tokens"], a["d"], a["rot"], a["cos"], a["sin"], a["rows"], a["pos"], a["ld_pos"], a["axes"],
                       a["axis"], a["flags"], None)


@pytest.mark.parametrize("kw,status,text", [
    (dict(count=0), A, "count=0"), (dict(count=9), A, "count=9"), (dict(d=12), U, "head_dim=12"),
    (dict(d=264), U, "head_dim=264"), (dict(d=0), U, "head_dim=0"), (dict(rot=8), U, "rot=8"),
    (dict(rot=144), U, "rot=144"), (dict(rot=0), U, "rot=0"), (dict(axes=0), U, "axes=0"), (dict(axes=5), U, "axes=5"),
    (dict(axes=1), A, "pair_axis[1]=1"), (dict(flags=2), A, "flags"), (dict(tokens=-1), A, "tokens=-1"),
    (dict(rows=0), A, "table_rows=0"), (dict(rows=1 << 31), A, "table_rows"), (dict(heads=0), A, "heads[0]=0"),
    (dict(ldx=248), A, "ldx[0]=248"), (dict(ldy=8), A, "ldy=8"), (dict(ldx=260), L, "multiples of 8"),
    (dict(x=None), A, "non-NULL"), (dict(y=None), A, "non-NULL"), (dict(x=P + 8), L, "aligned"),
    (dict(ldy=264), A, "in place"), (dict(cos=None), A, "non-NULL"), (dict(sin=P + 4), L, "aligned"),
    (dict(pos=None), A, "non-NULL"), (dict(pos=P + 2), L, "aligned"), (dict(ld_pos=2), A, "ld_pos=2"),
    (dict(tokens=1 << 40), U, "tokens"), (dict(heads=1 << 24, ldx=1 << 40, ldy=1 << 40, tokens=1 << 20), U, "too many"),
    (dict(ld_pos=1 << 62), U, "ld_pos"),
])
def test_bad_rope(lib, kw, status, text):
    assert rope(lib, **kw) == status, lib.wq_last_error()
    assert text in lib.wq_last_error().decode()


def test_rope_nothing_to_do(lib):
    assert rope(lib, tokens=0, x=None, y=None, cos=None, sin=None, pos=None) == dq.WQ_OK


def test_binding_refuses_host_tensors():
    with pytest.raises(ValueError, match="GPU tensor"):
        dq.KVCache(8, 64, 1, 16, torch.zeros((1, 1, 1024), dtype=torch.uint8), torch.zeros((1, 1, 1024), dtype=torch.uint8))
    with pytest.raises(ValueError, match="bits=5"):
        dq.KVCache(5, 64, 1, 16, None, None)
    with pytest.raises(ValueError, match="head_dim=0"):
        dq.KVCache(8, 0, 1, 16, None, None)


def test_native_binding_refuses_before_any_call():
    # the native half loads and asks its questions without a GPU
    c = dq.WqKvCache(8, 128, 2, 16, 10, P, P, P, P, None, 0)
    at, m = ctypes.addressof(c), dq._calls()
    x, i, f = torch.zeros((3, 256), dtype=torch.float16), torch.zeros(3, dtype=torch.int32), torch.zeros((4, 64))
    calls = [lambda: m.kv_write(at, x, x, i), lambda: m.kv_read(at, i, None), lambda: m.kv_read(at, i, (x, x)),
             lambda: m.attn_decode(at, x, i, i, None, 0, None, None, None),
             lambda: m.rope((x,), f, f, i, 128, None, False, None)]
    for call in calls:
        with pytest.raises(ValueError, match="GPU tensor"):
            call()
    with pytest.raises(TypeError, match="k must be a tensor, got list"):
        m.kv_write(at, [1], x, i)
    with pytest.raises(TypeError, match="4 arguments"):
        m.kv_write(at)
    with pytest.raises(ValueError, match="no cache"):
        m.kv_read(0, i, None)
    with pytest.raises(ValueError, match="arrays"):
        m.rope((), f, f, i, 128, None, False, None)
