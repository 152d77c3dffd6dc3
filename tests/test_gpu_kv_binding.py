"""What the Python calls of the cache, attention and rotary positions refuse
on the GPU: wrong types, shapes and strides as ValueError before anything is
launched, the library's own refusals as WqError with its message."""

import pytest
import torch

import dequant_gemv_rht_amd as dq

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def env():
    c = dq.KVCache.new(4, 16, 2, 128, 8)
    half = lambda *s: torch.zeros(s, dtype=torch.float16, device="cuda")   # noqa: E731
    ints = lambda *s: torch.zeros(s, dtype=torch.int32, device="cuda")     # noqa: E731
    return c, half, ints


def test_write_and_read_refuse(env):
    c, half, ints = env
    x, s = half(3, 256), ints(3)
    for args, text in (((x.float(), x, s), "float16"), ((x, half(3, 128), s), "channels"), ((x, x, ints(4)), "slots"),
                       ((x, x, s.long()), "int32"), ((half(256, 3).t(), x, s), "contiguous rows"),
                       ((half(3, 2, 128), x, s), "columns"), ((x, x, ints(3, 2)[:, 0]), "contiguous"), ((x.cpu(), x, s), "GPU")):
        with pytest.raises(ValueError, match=text):
            dq.wq_kv_write(c, *args)
    with pytest.raises(ValueError, match="channels"):
        dq.wq_kv_read(c, s, out=(x, half(3, 264)))
    with pytest.raises(ValueError, match="pair"):
        dq.wq_kv_read(c, s, out=(x,))
    with pytest.raises(dq.WqError, match="multiples of 8") as e:
        dq.wq_kv_write(c, half(3, 260)[:, :256], x, s)
    assert e.value.status == dq.WQ_E_ALIGN
    with pytest.raises(dq.WqError, match="aligned"):
        dq.wq_kv_read(c, s, out=(half(3, 264)[:, 4:260], x))


def test_attention_refuses(env):
    c, half, ints = env
    q, t, n = half(2, 512), ints(2, 4), ints(2)
    for args, kw, text in (((half(2, 500), t, n), {}, "heads of 128"), ((q, ints(3, 4), n), {}, "table"), ((q, t, ints(3)), {}, "lens"),
                           ((q, t.float(), n), {}, "int32"), ((q, ints(4, 2).t(), n), {}, "contiguous rows"),
                           ((q, t, n), dict(max_len=65), "max_len=65"), ((q, t, n), dict(out=half(2, 256)), "out"),
                           ((q, t, n), dict(workspace=torch.zeros(8)), "workspace")):
        with pytest.raises(ValueError, match=text):
            dq.wq_attn_decode(c, *args, **kw)
    with pytest.raises(dq.WqError, match="multiple of kv_heads") as e:
        dq.wq_attn_decode(c, half(2, 384), t, n)
    assert e.value.status == dq.WQ_E_ARG
    with pytest.raises(dq.WqError, match="window=-1"):
        dq.wq_attn_decode(c, q, t, n, window=-1)
    with pytest.raises(dq.WqError, match="scale"):
        dq.wq_attn_decode(c, q, t, n, scale=float("inf"))
    big, far = dq.KVCache.new(40, 16, 2, 128, 8), ints(2, 40)
    with pytest.raises(dq.WqError, match="workspace") as e:
        dq.wq_attn_decode(big, q, far, n, workspace=torch.zeros(16, dtype=torch.uint8, device="cuda"))
    assert e.value.status == dq.WQ_E_WORKSPACE
    with pytest.raises(TypeError):
        dq.wq_attn_decode(c, q, t, n, max_len="long")
    with pytest.raises(dq.WqError, match="max_len"):
        dq.wq_attn_decode_workspace(c, 1, 4, -1)


def test_rope_refuses(env):
    _, half, ints = env
    x, p = half(3, 256), ints(3)
    cos = torch.ones((8, 64), device="cuda")
    for args, kw, text in ((((x,), cos, cos[:4], p, 128), {}, "cos and sin"), (((x,), cos.half(), cos, p, 128), {}, "float32"),
                           (((x,), cos, cos, p.long(), 128), {}, "int32"), (((x,), cos, cos, ints(4), 128), {}, "heads"),
                           (((x,), cos, cos, p, 96), {}, "heads"), (((x,), cos, cos, p, 0), {}, "head_dim=0"),
                           (((x,), cos, cos, p, 128), dict(pair_axis=[0]), "pair_axis"), (((x,) * 9, cos, cos, p, 128), {}, "arrays"),
                           (((x,), cos, cos, p, 128), dict(out=(x, x)), "out"), (((x,), cos, cos, p, 128), dict(out=(half(3, 128),)), "out")):
        with pytest.raises(ValueError, match=text):
            dq.wq_rope(*args, **kw)
    with pytest.raises(dq.WqError, match="pair_axis") as e:
        dq.wq_rope((x,), cos, cos, p, 128, pair_axis=[1] * 64)
    assert e.value.status == dq.WQ_E_ARG
    with pytest.raises(dq.WqError, match="rot="):
        dq.wq_rope((x,), cos[:, :60].contiguous(), cos[:, :60].contiguous(), p, 128)


def test_results_are_what_was_asked_for(env):
    c, half, ints = env
    k, v = dq.wq_kv_read(c, ints(5))
    assert k.shape == v.shape == (5, 256) and k.dtype == torch.float16 and k.data_ptr() != v.data_ptr()
    ok, ov = half(5, 256), half(5, 256)
    a, b = dq.wq_kv_read(c, ints(5), out=[ok, ov])
    assert a.data_ptr() == ok.data_ptr() and b.data_ptr() == ov.data_ptr()
    y = half(2, 512)
    assert dq.wq_attn_decode(c, half(2, 512), ints(2, 4), ints(2), out=y) is y
    cos = torch.ones((8, 64), device="cuda")
    r = dq.wq_rope([half(3, 256), half(3, 128)], cos, cos, ints(3), 128)
    assert [t.shape for t in r] == [(3, 256), (3, 128)]
