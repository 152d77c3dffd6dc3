"""The attention side of a decoder block on a paged, quantised key-value cache: what is measured.

Four operators, each in its plain form (elementary torch operations in 32
bits) and, with ``own`` set, as the calls a user makes of the library:

* ``write``: new tokens' keys and values, quantised into the cache's pages
  (``wq_kv_write``), then the same rows read back (``wq_kv_read``), so that
  what the cache now holds comes out as the values it stands for;
* ``read``: cached rows read back as fp16 (``wq_kv_read``);
* ``attend``: attention of one new token per sequence over its pages
  (``wq_attn_decode``);
* ``rope``: rotary positions with one or several axes on queries and keys
  (``wq_rope``).

The cache (one layer).  ``bits`` is 4, 8 (codes with an fp16 scale and zero
per token and head, value = (code - zero) * scale) or 16 (fp16 values).  A
row is ``head_dim`` values, ``row`` bytes.  Arrays:

* ``k``: [pages][kv_heads][page_size * row bytes].  Within a page and head,
  16 tokens at a time: the block's rows cut into panels of min(64, row)
  bytes, [panel][16 tokens][panel bytes].
* ``v``: the same size; 4 tokens at a time, the four tokens' elements next
  to each other: [unit][4 tokens], a unit being one value (fp16, 8 bits) or
  the byte of two neighbouring 4-bit codes (even channel in the low half).
* ``k_params``, ``v_params``: fp16 [pages][kv_heads][page_size][2], scale
  and zero of each row.

With ``rotated`` the cache holds R x, R the block-128 random Hadamard
rotation with one sign per key-value channel: queries are rotated alike,
and what attention or a read gives out is rotated back.
"""

import math

import torch

own = False

GOLDEN = 0.6180339887498949


# ---------------------------------------------------------------- the cases

def _attend(name, seqs, q_heads, kv_heads, head_dim, max_len, page, bits, rotated, ragged, window=0):
    return {"name": name, "kind": "attend", "seqs": seqs, "q_heads": q_heads, "kv_heads": kv_heads,
            "head_dim": head_dim, "max_len": max_len, "page": page, "bits": bits, "rotated": rotated,
            "ragged": ragged, "window": window}


def _rows(name, kind, tokens, kv_heads, head_dim, page, bits, rotated, runs):
    return {"name": name, "kind": kind, "tokens": tokens, "kv_heads": kv_heads, "head_dim": head_dim,
            "page": page, "bits": bits, "rotated": rotated, "runs": runs}


def _rope(name, tokens, q_heads, kv_heads, head_dim, rot, axes, adjacent):
    return {"name": name, "kind": "rope", "tokens": tokens, "q_heads": q_heads, "kv_heads": kv_heads,
            "head_dim": head_dim, "rot": rot, "axes": axes, "adjacent": adjacent}


def listed():
    """32 query heads over 8 key-value heads of 128 are the widths of the
    decoder block's projections (4096 and 1024 channels)."""
    return [
        # one user, the first tokens of an answer: latency counts
        _attend("attend_first_tokens", 1, 32, 8, 128, 77, 16, 8, True, False),
        # one user with a long document
        _attend("attend_one_long", 1, 32, 8, 128, 32001, 64, 8, True, False),
        # a serving batch of conversations of every length, 4-bit cache, small pages
        _attend("attend_batch_ragged", 64, 32, 8, 128, 4099, 16, 4, True, True),
        # an unquantised cache, as many key-value heads as query heads, narrow heads
        _attend("attend_fp16_narrow", 16, 16, 16, 64, 2051, 32, 16, False, True),
        # wide heads, few of them, attention to the last 4000 positions only
        _attend("attend_wide_window", 24, 16, 2, 256, 8190, 128, 8, False, True, 4000),
        # a full card: long contexts in a large batch
        _attend("attend_largest", 64, 32, 8, 128, 16381, 64, 8, True, False),
        # a decode step's new tokens, one per sequence, each in a page of its own
        _rows("write_step", "write", 64, 8, 128, 16, 4, True, 64),
        # a prompt's keys and values
        _rows("write_prompt", "write", 8191, 8, 128, 64, 8, True, 1),
        # a cached prefix shared by a few new requests, back as fp16
        _rows("read_prefix", "read", 517, 8, 128, 16, 8, True, 4),
        # everything a long conversation holds, from a 4-bit cache
        _rows("read_long", "read", 30011, 8, 128, 64, 4, True, 1),
        # a decode step's queries and keys, text positions
        _rope("rope_step", 16, 32, 8, 128, 128, 1, False),
        # a prompt with images or video: time, height and width
        _rope("rope_video", 6001, 32, 8, 128, 128, 3, False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(("attend", "attend", "attend", "write", "write", "read", "rope"))
    head_dim = rng.choice((64, 128, 128, 256))
    kv_heads = rng.choice((1, 2, 4, 8))
    bits = rng.choice((4, 8, 8, 16))
    page = rng.choice((16, 32, 64, 128))
    rotated = head_dim >= 128 and bits < 16 and rng.random() < 0.6
    if kind == "attend":
        group = rng.choice((1, 2, 4, 5, 7, 8, 16))
        max_len = _log(rng, 1, 32768)
        room = 500_000_000 // (kv_heads * head_dim * max_len)
        seqs = _log(rng, 1, max(1, min(128, room)))
        window = _log(rng, 16, 8192) if rng.random() < 0.2 else 0
        c = _attend("", seqs, kv_heads * group, kv_heads, head_dim, max_len, page, bits, rotated,
                    rng.random() < 0.6, window)
    elif kind == "rope":
        rot = rng.choice((head_dim, head_dim, head_dim // 2))
        c = _rope("", _log(rng, 1, 8192), kv_heads * rng.choice((1, 2, 4)), kv_heads, head_dim, rot,
                  rng.choice((1, 2, 3)), rng.random() < 0.4)
    else:
        tokens = _log(rng, 1, 16384 if kind == "write" else 32768)
        c = _rows("", kind, tokens, kv_heads, head_dim, page, bits, rotated,
                  max(1, min(tokens, rng.choice((1, 4, 64, tokens)))))
    del c["name"]
    return c


def _lens(c):
    """The sequences' lengths: all max_len, or spread evenly over 1 .. max_len, the first the longest."""
    if not c["ragged"]:
        return [c["max_len"]] * c["seqs"]
    return [c["max_len"]] + [1 + int(c["max_len"] * math.modf(0.5 + i * GOLDEN)[0]) for i in range(1, c["seqs"])]


def _row_bytes(c):
    return c["head_dim"] * c["bits"] // 8


def work(c):
    if c["kind"] == "attend":
        seen = sum(min(n, c["window"] or n) for n in _lens(c))
        per = 2 * (_row_bytes(c) + (4 if c["bits"] < 16 else 0)) * c["kv_heads"]
        pages = sum(-(-min(n, c["window"] or n) // c["page"]) for n in _lens(c))
        return {"bytes": seen * per + 4 * pages + c["seqs"] * (4 + 4 * c["q_heads"] * c["head_dim"]),
                "flops": 4 * seen * c["q_heads"] * c["head_dim"]}
    if c["kind"] == "rope":
        n = c["tokens"] * (c["q_heads"] + c["kv_heads"])
        return {"bytes": 4 * n * c["head_dim"] + c["tokens"] * (4 * c["axes"] + 4 * c["rot"]),
                "flops": 3 * n * c["rot"]}
    n = c["tokens"] * c["kv_heads"]
    values, cached = 4 * n * c["head_dim"], 2 * n * (_row_bytes(c) + (4 if c["bits"] < 16 else 0))
    flops = 2 * n * c["head_dim"] * ((7 if c["rotated"] else 0) + 2)
    if c["kind"] == "write":
        return {"bytes": 2 * values + cached + 4 * c["tokens"], "flops": 2 * flops}
    return {"bytes": values + cached + 4 * c["tokens"], "flops": flops}


# ---------------------------------------------------------------- the inputs

def _normal(g, *shape):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32)


def _quantise(x, bits):
    """fp32 rows -> codes (as fp32), scale and zero (fp16): round to nearest
    over the row's range with 0 in it."""
    qmax = torch.full_like(x[..., :1], 2 ** bits - 1)
    lo = x.amin(-1, keepdim=True).clamp(max=0.0)
    hi = x.amax(-1, keepdim=True).clamp(min=0.0)
    scale = ((hi - lo) / qmax).clamp(max=65504.0).half()
    scale = torch.where(scale == 0, torch.ones_like(scale), scale)
    s = scale.float()
    zero = torch.minimum(torch.round(-lo / s).clamp(min=0.0), qmax)
    codes = torch.minimum(torch.round(x / s + zero).clamp(min=0.0), qmax)
    return codes, scale[..., 0], zero[..., 0].half()


def _pack(codes, bits):
    """Codes [..., head_dim] -> a row's units: fp16 values, or bytes (4 bits: two codes each)."""
    if bits == 16:
        return codes.half()
    codes = codes.to(torch.uint8)
    return codes if bits == 8 else codes[..., 0::2] | (codes[..., 1::2] << 4)


def _panel(units, bits):
    return min(32 if bits == 16 else 64, units)


def _cache(c, g, pages):
    """A filled cache of `pages` pages: normal keys (a few strong channels
    where nothing rotates them away) and values."""
    h, d, page, bits = c["kv_heads"], c["head_dim"], c["page"], c["bits"]
    x = _normal(g, pages, h, page, d)
    if not c["rotated"]:
        x[..., :: max(1, d // 4)] *= 4.0
    out = {"bits": bits, "head_dim": d, "kv_heads": h, "page": page}
    for name in ("k", "v"):
        if bits == 16:
            units = x.half()
            out[name + "_params"] = None
        else:
            codes, scale, zero = _quantise(x, bits)
            out[name + "_params"] = torch.stack((scale, zero), -1).contiguous()
            units = _pack(codes, bits)
        n = units.shape[-1]
        if name == "k":
            p = _panel(n, bits)
            units = units.view(pages, h, page // 16, 16, n // p, p).transpose(3, 4)
            x = _normal(g, pages, h, page, d)
        else:
            units = units.view(pages, h, page // 4, 4, n).transpose(3, 4)
        out[name] = units.reshape(pages, h, page * n).contiguous()
    out["signs"] = (torch.randint(-2 ** 31, 2 ** 31, (h * d // 32,), generator=g, device="cuda").to(torch.int32)
                    if c["rotated"] else None)
    return out


def prepare(c, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    s = {"kind": c["kind"]}
    d = c["head_dim"]
    if c["kind"] == "rope":
        t = c["tokens"]
        s["q"] = _normal(g, t, c["q_heads"] * d).half()
        s["k"] = _normal(g, t, c["kv_heads"] * d).half()
        step = torch.arange(t, device="cuda")
        start = torch.randint(0, 1000, (1,), generator=g, device="cuda")
        if c["axes"] == 1:
            pos = (start + step)[None]
        else:   # frames of 28 x 20 patches
            pos = torch.stack((start + step // 560, start + step % 560 // 28, start + step % 28))[: c["axes"]]
        s["positions"] = pos.to(torch.int32).contiguous()
        n = 1000 + t
        angle = (torch.arange(n, device="cuda", dtype=torch.float64)[:, None]
                 * 10000.0 ** (-torch.arange(0, c["rot"], 2, device="cuda", dtype=torch.float64) / c["rot"]))
        s["cos"], s["sin"] = angle.cos().float(), angle.sin().float()
        # pairs dealt to the axes in contiguous sections
        s["pair_axis"] = [i * c["axes"] // (c["rot"] // 2) for i in range(c["rot"] // 2)]
        s["axis_of"] = torch.tensor(s["pair_axis"], device="cuda")
        s["head_dim"], s["adjacent"] = d, c["adjacent"]
        return s
    if c["kind"] == "attend":
        lens = _lens(c)
        each = -(-c["max_len"] // c["page"])
        pages = c["seqs"] * each + 3
        s["cache"] = _cache(c, g, pages)
        s["q"] = (1.5 * _normal(g, c["seqs"], c["q_heads"] * d)).half()
        order = torch.randperm(pages, generator=g, device="cuda")[: c["seqs"] * each]
        s["table"] = order.view(c["seqs"], each).to(torch.int32).contiguous()
        s["lens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
        s["max_len"], s["window"], s["scale"] = c["max_len"], c["window"], d ** -0.5
        return s
    t, runs, page = c["tokens"], c["runs"], c["page"]
    # `runs` sequences of tokens, each at a place of its own in its first page
    each = -(-t // runs)
    per_run = each // page + 2
    s["cache"] = _cache(c, g, runs * per_run)
    order = torch.randperm(runs * per_run, generator=g, device="cuda").view(runs, per_run)
    first = torch.randint(0, page, (runs, 1), generator=g, device="cuda")
    at = first + torch.arange(each, device="cuda")
    slots = order.gather(1, at // page) * page + at % page
    s["slots"] = slots.reshape(-1)[:t].to(torch.int32).contiguous()
    if c["kind"] == "write":
        s["new_k"] = _normal(g, t, c["kv_heads"] * d)
        s["new_k"].view(t, c["kv_heads"], d)[..., :: max(1, d // 4)] *= 4.0
        s["new_k"] = s["new_k"].half()
        s["new_v"] = _normal(g, t, c["kv_heads"] * d).half()
    return s


# ---------------------------------------------------------------- the plain forms

def _stage(x, h):
    y = x.unflatten(-1, (-1, 2, h))
    a, b = y[..., 0, :], y[..., 1, :]
    return torch.stack((a + b, a - b), -2).flatten(-3)


def _hadamard(x):
    """The block-128 transform without its signs: seven steps of sums and differences, then 1/sqrt(128)."""
    shape = x.shape
    x = x.reshape(*shape[:-1], -1, 128)
    x = _stage(_stage(_stage(_stage(_stage(_stage(_stage(x, 1), 2), 4), 8), 16), 32), 64)
    return (x * 0.08838834764831845).reshape(shape)


def _sign(cache):
    """+-1 per key-value head and channel."""
    bit = torch.arange(32, device="cuda", dtype=torch.int32)
    bits = (cache["signs"][:, None] >> bit) & 1
    return (1.0 - 2.0 * bits.float()).view(cache["kv_heads"], cache["head_dim"])


def _values(units, params, bits):
    """A row's units -> fp32 values."""
    if bits == 16:
        return units.float()
    if bits == 4:
        units = torch.stack((units & 15, units >> 4), -1).flatten(-2)
    return (units.float() - params[..., 1:].float()) * params[..., :1].float()


def _pages_out(cache, name, pages):
    """The given pages' rows: fp32 [..., kv_heads, page, head_dim]."""
    bits, page = cache["bits"], cache["page"]
    x = cache[name][pages]
    lead, n = x.shape[:-1], x.shape[-1] // page
    if name == "k":
        p = _panel(n, bits)
        x = x.view(*lead, page // 16, n // p, 16, p).transpose(-3, -2)
    else:
        x = x.view(*lead, page // 4, n, 4).transpose(-2, -1)
    params = cache[name + "_params"]
    return _values(x.reshape(*lead, page, n), None if params is None else params[pages], bits)


def _places(cache, name, slots, n):
    """Where a row's n units are: its page [tokens, 1] and their places in the page [tokens, n]."""
    page, at = slots.long() // cache["page"], slots.long() % cache["page"]
    unit = torch.arange(n, device="cuda")
    if name == "k":
        p = _panel(n, cache["bits"])
        place = (at // 16 * 16 * n)[:, None] + unit // p * (16 * p) + (at % 16 * p)[:, None] + unit % p
    else:
        place = (at // 4 * 4 * n)[:, None] + unit * 4 + (at % 4)[:, None]
    return page, at, place


def _plain_read(cache, slots):
    out = []
    n = cache["k"].shape[-1] // cache["page"]
    head = torch.arange(cache["kv_heads"], device="cuda")[None, :, None]
    for name in ("k", "v"):
        page, at, place = _places(cache, name, slots, n)
        units = cache[name][page[:, None, None], head, place[:, None, :]]
        params = cache[name + "_params"]
        x = _values(units, None if params is None else params[page, :, at], cache["bits"])
        if cache["signs"] is not None:
            x = _hadamard(x) * _sign(cache)
        out.append(x.half().flatten(1))
    return out


def _plain_write(cache, k, v, slots):
    head = torch.arange(cache["kv_heads"], device="cuda")[None, :, None]
    for name, x in (("k", k), ("v", v)):
        x = x.float().view(len(slots), cache["kv_heads"], cache["head_dim"])
        if cache["signs"] is not None:
            x = _hadamard(x * _sign(cache))
        if cache["bits"] < 16:
            x, scale, zero = _quantise(x, cache["bits"])
        units = _pack(x, cache["bits"])
        page, at, place = _places(cache, name, slots, units.shape[-1])
        cache[name][page[:, None, None], head, place[:, None, :]] = units
        if cache["bits"] < 16:
            cache[name + "_params"][page, :, at] = torch.stack((scale, zero), -1)


def _plain_attend(s):
    cache, q, table = s["cache"], s["q"], s["table"].long()
    b, h, d = q.shape[0], cache["kv_heads"], cache["head_dim"]
    q = q.float().view(b, h, -1, d)
    if cache["signs"] is not None:
        q = _hadamard(q * _sign(cache)[:, None])
    # [b, pages, h, page, d] -> [b, h, positions, d]
    k = _pages_out(cache, "k", table).transpose(1, 2).flatten(2, 3)
    score = torch.matmul(q, k.transpose(-1, -2)) * s["scale"]
    del k
    at = torch.arange(score.shape[-1], device="cuda")
    length = s["lens"].long()[:, None]
    seen = at < length
    if s["window"]:
        seen = seen & (at >= length - s["window"])
    seen = seen[:, None, None]
    top = torch.where(seen, score, torch.full_like(score, -math.inf)).amax(-1, keepdim=True)
    p = torch.where(seen, torch.exp(score - top), torch.zeros_like(score))
    total = p.sum(-1, keepdim=True)
    v = _pages_out(cache, "v", table).transpose(1, 2).flatten(2, 3)
    y = torch.matmul(p, v) / torch.where(total > 0, total, torch.ones_like(total))
    if cache["signs"] is not None:
        y = _hadamard(y) * _sign(cache)[:, None]
    return y.reshape(b, -1).half()


def _plain_rope(s):
    half = len(s["pair_axis"])
    pos = s["positions"].long()[s["axis_of"]].t()
    pair = torch.arange(half, device="cuda")
    cos, sin = s["cos"][pos, pair][:, None], s["sin"][pos, pair][:, None]
    out = []
    for x in (s["q"], s["k"]):
        y = x.float().view(x.shape[0], -1, s["head_dim"])
        rot, rest = y[..., : 2 * half], y[..., 2 * half:]
        if s["adjacent"]:
            a, b = rot[..., 0::2], rot[..., 1::2]
            rot = torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2)
        else:
            a, b = rot[..., :half], rot[..., half:]
            rot = torch.cat((a * cos - b * sin, b * cos + a * sin), -1)
        out.append(torch.cat((rot, rest), -1).flatten(1).half())
    return out


def run(s):
    if own:
        return _own(s)
    if s["kind"] == "attend":
        return _plain_attend(s)
    if s["kind"] == "rope":
        return _plain_rope(s)
    if s["kind"] == "write":
        _plain_write(s["cache"], s["new_k"], s["new_v"], s["slots"])
    return _plain_read(s["cache"], s["slots"])


# ---------------------------------------------------------------- the library's calls

def _own(s):
    import dequant_gemv_rht_amd as dq

    if s["kind"] == "rope":
        return dq.wq_rope((s["q"], s["k"]), s["cos"], s["sin"], s["positions"], s["head_dim"],
                          pair_axis=s["pair_axis"], adjacent=s["adjacent"])
    c = s["cache"]
    cache = s.get("handle")
    if cache is None:
        cache = s["handle"] = dq.KVCache(c["bits"], c["head_dim"], c["kv_heads"], c["page"], c["k"], c["v"],
                                         c["k_params"], c["v_params"], c["signs"])
    if s["kind"] == "attend":
        return dq.wq_attn_decode(cache, s["q"], s["table"], s["lens"], max_len=s["max_len"], window=s["window"],
                                 scale=s["scale"])
    if s["kind"] == "write":
        dq.wq_kv_write(cache, s["new_k"], s["new_v"], s["slots"])
    return dq.wq_kv_read(cache, s["slots"])


# ---------------------------------------------------------------- from the definition, in 64 bits

def _exact_rotation(signs, heads, d):
    """R of every key-value head: fp64 [heads][d][d], from the popcount formula."""
    i = torch.arange(d, device="cuda")
    both = i[:, None] & i[None] & 127
    odd = torch.zeros_like(both)
    for b in range(7):
        odd ^= (both >> b) & 1
    m = torch.where((i[:, None] // 128) == (i[None] // 128), 1.0 - 2.0 * odd.double(), 0.0) / math.sqrt(128.0)
    channel = torch.arange(heads * d, device="cuda")
    word = signs.long()[channel // 32]
    flip = (1.0 - 2.0 * ((word >> (channel % 32)) & 1).double()).view(heads, 1, d)
    return m[None] * flip


def _exact_rows(cache, name, slots):
    """Rows by slot as fp64 [rows][heads][d]: each value from its own bits, wherever the layout puts them."""
    d, bits, size = cache["head_dim"], cache["bits"], cache["page"]
    page, at = slots // size, slots % size
    ch = torch.arange(d, device="cuda")[None]
    unit = ch // 2 if bits == 4 else ch
    n = d // 2 if bits == 4 else d
    if name == "k":
        p = min(n, 32 if bits == 16 else 64)
        place = ((at[:, None] // 16) * (n // p) + unit // p) * 16 * p + (at[:, None] % 16) * p + unit % p
    else:
        place = ((at[:, None] // 4) * n + unit) * 4 + at[:, None] % 4
    flat = cache[name].reshape(cache[name].shape[0], cache["kv_heads"], -1)
    got = flat[page[:, None], :, place].permute(0, 2, 1)   # [rows][heads][d]
    if bits == 16:
        return got.double()
    code = got.long()
    if bits == 4:
        code = (code >> (4 * (ch % 2))) & 15
    par = cache[name + "_params"][page, :, at].double()
    return (code.double() - par[..., 1:]) * par[..., :1]


def exact(c, seed):
    s = prepare(c, seed)
    d = c["head_dim"]
    if c["kind"] == "rope":
        half = c["rot"] // 2
        i = torch.arange(half, device="cuda")
        first, second = (2 * i, 2 * i + 1) if c["adjacent"] else (i, i + half)
        where = s["positions"].long()[torch.tensor(s["pair_axis"], device="cuda")]   # [half][tokens]
        cos, sin = (s[n].double()[where, i[:, None]].t()[:, None] for n in ("cos", "sin"))
        out = []
        for x in (s["q"], s["k"]):
            y = x.double().view(c["tokens"], -1, d)
            z = y.clone()
            z[..., first] = y[..., first] * cos - y[..., second] * sin
            z[..., second] = y[..., second] * cos + y[..., first] * sin
            out.append(z.flatten(1))
        return out
    cache, h = s["cache"], c["kv_heads"]
    r = _exact_rotation(cache["signs"], h, d) if c["rotated"] else None
    if c["kind"] == "attend":
        q = s["q"].double().view(c["seqs"], h, -1, d)
        if r is not None:
            q = torch.stack([q[:, i] @ r[i].t() for i in range(h)], 1)
        out = torch.zeros_like(q)
        for b, n in enumerate(_lens(c)):
            pos = torch.arange(max(0, n - c["window"]) if c["window"] else 0, n, device="cuda")
            slots = s["table"][b].long()[pos // c["page"]] * c["page"] + pos % c["page"]
            k = _exact_rows(cache, "k", slots).permute(1, 2, 0).contiguous()
            w = torch.softmax(torch.bmm(q[b], k) * s["scale"], -1)
            out[b] = torch.bmm(w, _exact_rows(cache, "v", slots).permute(1, 0, 2).contiguous())
        if r is not None:
            out = torch.stack([out[:, i] @ r[i] for i in range(h)], 1)
        return out.reshape(c["seqs"], -1)
    out = []
    for name in ("k", "v"):
        if c["kind"] == "read":
            x = _exact_rows(cache, name, s["slots"].long())
        else:
            x = s["new_" + name].double().view(c["tokens"], h, d)
            if r is not None:
                x = torch.stack([x[:, i] @ r[i].t() for i in range(h)], 1)
            if c["bits"] < 16:
                top = float(2 ** c["bits"] - 1)
                lo, hi = x.amin(-1, True).clamp(max=0), x.amax(-1, True).clamp(min=0)
                scale = ((hi - lo) / top).clamp(max=65504.0).half().double()
                scale[scale == 0] = 1.0
                zero = torch.round(-lo / scale).clamp(0, top)
                x = (torch.round(x / scale + zero).clamp(0, top) - zero) * scale
        if r is not None:
            x = torch.stack([x[:, i] @ r[i] for i in range(h)], 1)
        out.append(x.flatten(1))
    return out
