"""KVCache hands the library what its tensors are now: assigning a tensor, or
moving one's storage, must never leave a call with memory that was freed."""

import pytest
import torch

import dequant_gemv_rht_amd as dq

FIELDS = ("k", "v", "k_params", "v_params")


def arrays(pages, device, bits=8, heads=2, page=16, d=64):
    units = d // 2 if bits == 4 else d
    dt = torch.float16 if bits == 16 else torch.uint8
    k, v = (torch.zeros((pages, heads, page * units), dtype=dt, device=device) for _ in range(2))
    if bits == 16:
        return dict(k=k, v=v)
    kp, vp = (torch.zeros((pages, heads, page, 2), dtype=torch.float16, device=device) for _ in range(2))
    return dict(k=k, v=v, k_params=kp, v_params=vp)


def grow(cache, new):
    for name, t in new.items():
        setattr(cache, name, t)


@pytest.mark.parametrize("bits", [4, 8, 16])
def test_descriptor_follows_assignment(monkeypatch, bits):
    # CPU: the descriptor alone, with host tensors let through
    monkeypatch.setattr(dq, "_dev", lambda t, dtype, name: t)
    cache = dq.KVCache(bits, 64, 2, 16, **arrays(3, "cpu", bits))
    assert cache._c.pages == 3 and cache._c.k == cache.k.data_ptr()
    new = arrays(7, "cpu", bits)
    grow(cache, new)
    assert cache._c.pages == 7
    for name, t in new.items():
        assert getattr(cache._c, name) == t.data_ptr()
    # arrays that do not belong together are refused at the next use
    cache.v = arrays(5, "cpu", bits)["v"]
    with pytest.raises(ValueError, match="v: "):
        cache._c
    cache.v = new["v"]
    cache.head_dim = 96
    with pytest.raises(ValueError, match="head_dim=96"):
        cache._c
    cache.head_dim = 64
    assert cache._c.v == new["v"].data_ptr()


@pytest.mark.gpu
@pytest.mark.parametrize("bits", [4, 8, 16])
def test_calls_follow_assignment(bits):
    cache = dq.KVCache(bits, 64, 2, 16, **arrays(2, "cuda", bits))
    old = {n: getattr(cache, n) for n in FIELDS}
    gen = torch.Generator(device="cuda")
    gen.manual_seed(bits)
    x, y = (torch.randn((5, 128), generator=gen, device="cuda").half() for _ in range(2))
    slots = torch.tensor([16, 17, 18, 19, 31], dtype=torch.int32, device="cuda")
    dq.wq_kv_write(cache, x, y, slots)
    before = {n: None if t is None else t.clone() for n, t in old.items()}
    first = dq.wq_kv_read(cache, slots)
    # grown, as a server does: more pages, the old ones' contents in front
    new = arrays(6, "cuda", bits)
    for n, t in new.items():
        t[:2].copy_(old[n])
    grow(cache, new)
    far = slots + 64
    dq.wq_kv_write(cache, y, x, far)
    for a, b in zip(dq.wq_kv_read(cache, torch.cat([slots, far])), (first[0], first[1])):
        assert torch.equal(a[:5], b)
    a, b = dq.wq_kv_read(cache, far)
    assert torch.equal(a, first[1]) and torch.equal(b, first[0])
    q = torch.randn((1, 256), generator=gen, device="cuda").half()
    table = torch.tensor([[5]], dtype=torch.int32, device="cuda")
    one = torch.ones(1, dtype=torch.int32, device="cuda")
    dq.wq_kv_write(cache, x[:1], y[:1], table[0] * 16)
    k, v = dq.wq_kv_read(cache, table[0] * 16)
    got = dq.wq_attn_decode(cache, q, table, one)
    assert torch.allclose(got.view(2, 2, 64).float(), v.view(2, 1, 64).expand(2, 2, 64).float(), rtol=2e-3, atol=1e-4)
    assert dq.wq_attn_decode_workspace(cache, 1, 4, 96) >= 0
    for n, t in old.items():
        assert t is None or torch.equal(t, before[n])


@pytest.mark.gpu
def test_moved_storage_is_followed_and_resized_refused():
    cache = dq.KVCache(8, 64, 2, 16, **arrays(2, "cuda"))
    gen = torch.Generator(device="cuda")
    gen.manual_seed(1)
    x = torch.randn((4, 128), generator=gen, device="cuda").half()
    slots = torch.arange(4, dtype=torch.int32, device="cuda")
    was = cache.k.clone()
    cache.k.set_(was)                         # the same tensor, another storage
    dq.wq_kv_write(cache, x, x, slots)
    assert was.any() and torch.equal(dq.wq_kv_read(cache, slots)[0], dq.wq_kv_read(cache, slots)[1])
    # a tensor of another size under the cache's name: refused, whichever it is
    for name in FIELDS:
        dq.wq_kv_write(cache, x, x, slots)    # described as it is now
        t = getattr(cache, name)
        keep = t.clone()
        t.resize_((1, *t.shape[1:]))
        for call in (lambda: dq.wq_kv_write(cache, x, x, slots), lambda: dq.wq_kv_read(cache, slots),
                     lambda: dq.wq_attn_decode(cache, x, slots[:, None].contiguous(), slots)):
            with pytest.raises(ValueError, match=f"{name}.*KVCache"):
                call()
        setattr(cache, name, keep)
