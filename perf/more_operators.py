"""What a serving step of many requests does around the projections and the attention: what is measured.

Three operators, each in its plain form (elementary torch operations) and,
with ``own`` set, as the calls a user makes of the library:

* ``slots``: pages, cache slots and positions for the tokens that a step adds
  to its sequences, from their lengths (``wq_kv_slots``);
* ``lora``: the low-rank adapters of many requests beside shared projections,
  y = base + scale B (A x) with the adapter of each row (``wq_lora``);
* ``sample``: the next token of each row of logits under a temperature, top-k,
  top-p and min-p of its own, from given random numbers (``wq_sample``).

Slots.  Sequence s holds ``lens[s]`` tokens and gets ``new[s]`` more; page j of
a sequence is ``table[s][j]``.  Pages that the new tokens need are the next
ones of ``free`` from place ``used`` on, in the sequences' order.  A sequence
is served if its rows end within the step's ``tokens`` rows, its pages fit its
row of the table, and the pages that it and those before it need are there.
Rows of the step that belong to no served sequence have -1 everywhere.

Sampling.  w = exp((logit - max) / T).  By falling logit, equal ones by rising
index: the first ``top_k``; of these, those before which less than ``top_p`` of
their sum lies; of these, those with w >= ``min_p``.  The token is the first by
index where the sum of the kept w passes u times all of it.  T = 0 is the
largest logit.  A row without a finite logit gives -1.
"""

import math

import numpy as np
import torch

own = False

# the projections of the decoder block, input -> outputs; those with one input share it
SETS = {
    "single": [(1024, [512])],
    "qkv": [(2560, [4096, 1024, 1024])],
    "o": [(4096, [2560])],
    "gate_up": [(2560, [9728, 9728])],
    "down": [(9728, [2560])],
    "block": [(2560, [4096, 1024, 1024]), (4096, [2560]), (2560, [9728, 9728]), (9728, [2560])],
}


# ---------------------------------------------------------------- the cases

def _slots(name, seqs, page, held, prompts, prompt, pad, short=False):
    return {"name": name, "kind": "slots", "seqs": seqs, "page": page, "held": held, "prompts": prompts,
            "prompt": prompt, "pad": pad, "short": short}


def _lora(name, projections, rows, adapters, rank, order, bare=0, wide=False):
    return {"name": name, "kind": "lora", "set": projections, "rows": rows, "adapters": adapters, "rank": rank,
            "order": order, "bare": bare, "wide": wide}


def _sample(name, rows, vocab, mode, half=False, masked=False):
    return {"name": name, "kind": "sample", "rows": rows, "vocab": vocab, "mode": mode, "half": half,
            "masked": masked}


def listed():
    return [
        # a decode step: one new token for each conversation of a batch
        _slots("slots_step", 64, 16, 4000, 0, 0, 0),
        # a few prompts arrive at once, padded to a captured graph's rows
        _slots("slots_prompts", 9, 64, 0, 9, 2047, 500),
        # a full server: a thousand conversations, prompts among them
        _slots("slots_largest", 1024, 16, 8000, 60, 1500, 0),
        # one user with an adapter on the attention's inputs: latency counts
        _lora("lora_one", "qkv", 1, 4, 16, "scattered"),
        # a serving batch, half of it sharing adapters, some rows without one
        _lora("lora_batch", "gate_up", 64, 28, 16, "scattered", 8),
        # every request with an adapter of its own, on the whole block
        _lora("lora_largest", "block", 128, 128, 32, "scattered"),
        # a prompt step: three requests' rows one after another
        _lora("lora_prompt", "qkv", 4001, 3, 64, "runs"),
        # a narrow adapter on a long input, results in 32 bits
        _lora("lora_down_fp32", "down", 17, 5, 8, "scattered", 2, True),
        # one user's answer: the usual settings on the head's logits
        _sample("sample_one", 1, 151936, "usual"),
        # a serving batch in which every request has settings of its own
        _sample("sample_batch", 64, 151936, "mixed"),
        # a small vocabulary in 16 bits (many equal logits), some rows held to a grammar
        _sample("sample_fp16_masked", 33, 32003, "mixed", True, True),
        # a full card of requests
        _sample("sample_largest", 256, 151936, "mixed"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(("slots", "lora", "lora", "sample", "sample"))
    if kind == "slots":
        seqs = _log(rng, 1, 1024)
        prompts = rng.choice((0, rng.randint(0, min(seqs, 48))))
        c = _slots("", seqs, rng.choice((16, 32, 64, 128)), _log(rng, 1, 8000), prompts, _log(rng, 1, 1500),
                   rng.choice((0, rng.randint(1, 300))), rng.random() < 0.25)
    elif kind == "lora":
        projections = rng.choice(("single", "qkv", "o", "gate_up", "down", "block"))
        rank = rng.choice((8, 16, 16, 32, 64))
        order = rng.choice(("scattered", "scattered", "runs"))
        rows = _log(rng, 1, 128 if order == "scattered" else 4096)
        if projections in ("block", "gate_up") and order == "runs":
            rows = min(rows, 700)
        each = rank * sum(k + n for k, ns in SETS[projections] for n in ns)
        adapters = _log(rng, 1, max(1, min(128, 200_000_000 // each)) if order == "scattered" else 6)
        bare = rng.choice((0, 0, rng.randint(0, rows // 4)))
        c = _lora("", projections, rows, adapters, rank, order, bare, rng.random() < 0.3)
    else:
        vocab = _log(rng, 1000, 262144)
        rows = _log(rng, 1, max(1, min(256, 30_000_000 // vocab)))
        c = _sample("", rows, vocab, rng.choice(("usual", "mixed", "mixed", "open", "top_p", "top_k", "min_p")),
                    rng.random() < 0.35, rng.random() < 0.3)
    del c["name"]
    return c


def _new(c):
    """New tokens of each sequence: prompts of uneven lengths spread among single tokens (and none for some)."""
    seqs, prompts = c["seqs"], c["prompts"]
    new = [0 if prompts and i % 17 == 16 else 1 for i in range(seqs)]
    for j in range(prompts):
        new[j * seqs // prompts] = 1 + int(c["prompt"] * math.modf(0.5 + j * 0.6180339887498949)[0])
    return new


def _projections(c):
    return [(i, k, n) for i, (k, ns) in enumerate(SETS[c["set"]]) for n in ns]


def work(c):
    if c["kind"] == "slots":
        new = _new(c)
        total = sum(new)
        return {"bytes": 24 * c["seqs"] + 12 * (total + c["pad"]) + 8 * (total // c["page"]), "flops": 4 * total}
    if c["kind"] == "lora":
        rows = c["rows"] - c["bare"]
        used = min(rows, c["adapters"])
        size = 4 if c["wide"] else 2
        each = c["rank"] * sum(k + n for _, k, n in _projections(c))
        return {"bytes": 2 * used * each + c["rows"] * (4 + sum(2 * k for k, _ in SETS[c["set"]])
                                                        + 2 * size * sum(n for _, _, n in _projections(c))),
                "flops": 2 * rows * each}
    return {"bytes": c["rows"] * (c["vocab"] * (2 if c["half"] else 4) + 28), "flops": 4 * c["rows"] * c["vocab"]}


# ---------------------------------------------------------------- the inputs

def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _normal(g, *shape):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32)


def _uniform(g, *shape):
    return torch.rand(shape, generator=g, device="cuda", dtype=torch.float32)


def prepare(c, seed):
    g = _generator(seed)
    s = {"kind": c["kind"]}
    if c["kind"] == "slots":
        new = torch.tensor(_new(c), dtype=torch.int32, device="cuda")
        lens = torch.randint(0, c["held"] + 1, (c["seqs"],), generator=g, device="cuda").to(torch.int32)
        page = c["page"]
        wide = -(-(c["held"] + max(_new(c))) // page) + 1
        held = (lens.long() + page - 1) // page
        need = int(((lens.long() + new + page - 1) // page - held).sum())
        pages = int(held.sum()) + need + 7
        order = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
        s["table"] = torch.full((c["seqs"], wide), -1, dtype=torch.int32, device="cuda")
        first = torch.cumsum(held, 0) - held
        at = torch.arange(wide, device="cuda")
        own_pages = order[(first[:, None] + at).clamp(max=pages - 1)]
        s["table"] = torch.where(at < held[:, None], own_pages, s["table"]).contiguous()
        # the pages that no sequence holds; two of them are gone already
        s["free"] = order[int(held.sum()):].contiguous()
        s["used"] = torch.full((1,), 2, dtype=torch.int32, device="cuda")
        if c["short"]:   # a full cache: half of what is asked for
            s["free"] = s["free"][: 2 + need // 2].contiguous()
        s["lens"], s["new"], s["page"], s["pages"] = lens, new, page, pages
        s["tokens"] = sum(_new(c)) + c["pad"]
        return s
    if c["kind"] == "lora":
        rows, adapters, rank = c["rows"], c["adapters"], c["rank"]
        out = torch.float32 if c["wide"] else torch.float16
        x = [_normal(g, rows, k).half() for k, _ in SETS[c["set"]]]
        s["x"], s["a"], s["b"], s["base"] = [], [], [], []
        for i, k, n in _projections(c):
            s["x"].append(x[i])
            s["a"].append((_normal(g, adapters, rank, k) * k ** -0.5).half())
            s["b"].append((_normal(g, adapters, n, rank) * 0.1).half())
            s["base"].append(_normal(g, rows, n).to(out))
        s["scales"] = 0.25 + 1.75 * _uniform(g, adapters)
        with_one = rows - c["bare"]
        name = torch.randperm(adapters, generator=g, device="cuda")
        at = torch.arange(with_one, device="cuda")
        used = min(with_one, adapters)
        if c["order"] == "runs":
            ids = torch.cat((name[at * used // max(1, with_one)], at.new_full((c["bare"],), -1)))
        else:
            ids = torch.cat((name[at % max(1, used)], at.new_full((c["bare"],), -1)))
            ids = ids[torch.randperm(rows, generator=g, device="cuda")]
        s["ids"] = ids.to(torch.int32).contiguous()
        return s
    rows, vocab = c["rows"], c["vocab"]
    # rows from sure to open: most logits far below a few likely ones
    spread = 1.0 + 2.0 * _uniform(g, rows, 1)
    logits = spread * _normal(g, rows, vocab)
    likely = torch.randint(0, vocab, (rows, 12), generator=g, device="cuda")
    logits.scatter_add_(1, likely, 3.0 + 9.0 * _uniform(g, rows, 12))
    if c["masked"]:   # every third row may only answer with some 1 in 50 of the tokens
        shut = (torch.arange(rows, device="cuda") % 3 == 1)[:, None] & (_uniform(g, rows, vocab) > 0.02)
        logits = torch.where(shut, torch.full_like(logits, -math.inf), logits)
    s["logits"] = logits.half() if c["half"] else logits
    s["u"] = _uniform(g, rows)
    mode = c["mode"]
    row = torch.arange(rows, device="cuda")
    warm, k = 0.5 + 0.7 * _uniform(g, rows), torch.randint(1, 200, (rows,), generator=g, device="cuda")
    p, m = 0.8 + 0.19 * _uniform(g, rows), 0.02 + 0.1 * _uniform(g, rows)
    one, none = torch.ones_like(p), torch.zeros_like(m)
    if mode == "usual":
        s["temperature"], s["top_k"], s["top_p"], s["min_p"] = 0.7 * one, torch.full_like(k, 50), 0.9 * one, none
    elif mode == "mixed":   # rows in turn: greedy, open, top-k, top-p, both, all three
        kind = row % 6
        s["temperature"] = torch.where(kind == 0, none, warm)
        s["top_k"] = torch.where((kind == 2) | (kind >= 4), k, torch.zeros_like(k))
        s["top_p"] = torch.where(kind >= 3, p, one)
        s["min_p"] = torch.where(kind == 5, m, none)
    else:
        s["temperature"] = warm
        s["top_k"] = k if mode == "top_k" else torch.zeros_like(k)
        s["top_p"] = p if mode == "top_p" else one
        s["min_p"] = m if mode == "min_p" else none
    s["top_k"] = s["top_k"].to(torch.int32)
    return s


# ---------------------------------------------------------------- the plain forms

def _plain_slots(s):
    page, pages, tokens, seqs = s["page"], s["pages"], s["tokens"], s["lens"].shape[0]
    held = torch.clamp(s["lens"].long(), min=0)
    new = torch.clamp(s["new"].long(), min=0)
    end = torch.cumsum(new, 0)
    fits = (end <= tokens) & (held + new <= s["table"].shape[1] * page)
    old_pages = (held + page - 1) // page
    need = torch.where(fits, (held + new + page - 1) // page - old_pages, torch.zeros_like(held))
    last_page = torch.cumsum(need, 0)
    used = s["used"].long()
    room = s["free"].shape[0] - used
    served = fits & (need.eq(0) | (last_page <= room))
    first_page = used + last_page - need
    # the new pages in the table
    at = torch.arange(s["table"].shape[1], device="cuda")
    mine = served[:, None] & (at >= old_pages[:, None]) & (at < (old_pages + need)[:, None])
    place = (first_page - old_pages)[:, None] + at
    free = s["free"][place.clamp(0, s["free"].shape[0] - 1)]
    table = torch.where(mine, free, s["table"])
    # the rows of the step
    row = torch.arange(tokens, device="cuda")
    seq = torch.searchsorted(end, row, right=True)
    live = seq < seqs
    seq = seq.clamp(max=seqs - 1)
    live = live & served[seq]
    pos = held[seq] + row - (end - new)[seq]
    number = table[seq, (pos // page).clamp(0, table.shape[1] - 1)].long()
    none = torch.full_like(row, -1)
    slot = torch.where(live & (number >= 0) & (number < pages), number * page + pos % page, none)
    lens = torch.where(served, held + new, s["lens"].long())
    last = torch.where(served & (new > 0), end - 1, torch.full_like(end, -1))
    taken = torch.where(served, last_page, torch.zeros_like(last_page)).amax(0, keepdim=True)
    out = (slot, torch.where(live, pos, none), torch.where(live, seq, none), lens, last, used + taken)
    return [x.to(torch.int32) for x in out] + [table]


def _plain_lora(s):
    """All adapters' products, those of other adapters than a row's own left out between the two."""
    adapters = s["scales"].shape[0]
    mine = s["ids"].long()[:, None] == torch.arange(adapters, device="cuda")
    weight = torch.where(mine, s["scales"], torch.zeros_like(s["scales"]))
    out = []
    for x, a, b, base in zip(s["x"], s["a"], s["b"], s["base"]):
        t = torch.matmul(x.float(), a.float().flatten(0, 1).t()).unflatten(1, (adapters, -1)) * weight[:, :, None]
        y = torch.matmul(t.flatten(1), b.float().transpose(1, 2).flatten(0, 1))
        out.append((base.float() + y).to(base.dtype))
    return out


def _plain_sample(s):
    x = s["logits"].float()
    x = torch.where(torch.isnan(x), torch.full_like(x, -math.inf), x)
    rows, vocab = x.shape
    greedy = ~(s["temperature"] > 0)
    heat = torch.where(greedy, torch.ones_like(s["temperature"]), s["temperature"]).double()[:, None]
    top_k = torch.where(greedy, torch.ones_like(s["top_k"]), s["top_k"])
    top_k = torch.where((top_k <= 0) | (top_k > vocab), torch.full_like(top_k, vocab), top_k)[:, None]
    ordered, order = torch.sort(x, dim=1, descending=True, stable=True)
    top = ordered[:, :1].double()
    ordered = ordered.double()
    w = torch.where(ordered == top, torch.ones_like(ordered), torch.exp((ordered - top) / heat))
    w = torch.where(ordered == -math.inf, torch.zeros_like(w), w)
    rank = torch.arange(vocab, device="cuda")
    w = torch.where(rank < top_k, w, torch.zeros_like(w))
    up_to = torch.cumsum(w, 1)
    before = torch.cat((torch.zeros_like(up_to[:, :1]), up_to[:, :-1]), 1)
    top_p = s["top_p"].double()[:, None]
    keep = (before < top_p * up_to[:, -1:]) | (rank == 0) | (top_p >= 1)
    keep = keep & (w >= s["min_p"].clamp(max=1.0).double()[:, None])
    kept = torch.zeros_like(w).scatter(1, order, torch.where(keep, w, torch.zeros_like(w)))
    up_to = torch.cumsum(kept, 1)
    total = up_to[:, -1:]
    ids = (up_to <= s["u"].double()[:, None] * total).sum(1, keepdim=True)
    last = torch.where(kept > 0, rank, torch.zeros_like(rank)).amax(1, keepdim=True)
    ids = torch.minimum(ids, last)
    chance = torch.log(kept.gather(1, ids) / total)
    empty = total == 0
    ids = torch.where(empty, torch.full_like(ids, -1), ids)
    chance = torch.where(empty, torch.full_like(chance, -math.inf), chance)
    return [ids[:, 0].to(torch.int32), chance[:, 0].float()]


def run(s):
    if own:
        return _own(s)
    if s["kind"] == "slots":
        return _plain_slots(s)
    if s["kind"] == "lora":
        return _plain_lora(s)
    return _plain_sample(s)


# ---------------------------------------------------------------- the library's calls

def _own(s):
    import dequant_gemv_rht_amd as dq

    if s["kind"] == "slots":
        step = dq.wq_kv_slots(s["page"], s["pages"], s["table"], s["lens"], s["new"], s["free"], s["used"],
                              s["tokens"])
        return list(step) + [s["table"]]
    if s["kind"] == "lora":
        return list(dq.wq_lora(s["a"], s["b"], s["x"], s["ids"], s["base"], scales=s["scales"]))
    return list(dq.wq_sample(s["logits"], s["u"], temperature=s["temperature"], top_k=s["top_k"], top_p=s["top_p"],
                             min_p=s["min_p"]))


# ---------------------------------------------------------------- in 64 bits

def exact(c, seed):
    if c["kind"] == "slots":
        return None   # whole numbers
    s = prepare(c, seed)
    if c["kind"] == "lora":
        # adapter by adapter, over its own rows
        ids = s["ids"].cpu().numpy()
        out = [y.double() for y in s["base"]]
        for adapter in sorted(set(ids.tolist()) - {-1}):
            rows = torch.from_numpy(np.flatnonzero(ids == adapter)).cuda()
            factor = s["scales"][adapter].double()
            for y, x, a, b in zip(out, s["x"], s["a"], s["b"]):
                inner = x[rows].double() @ a[adapter].double().t()
                y[rows] += factor * (inner @ b[adapter].double().t())
        return out
    logits = s["logits"].float().cpu().numpy().astype(np.float64)
    heat, p, m, u = (s[n].cpu().numpy().astype(np.float64) for n in ("temperature", "top_p", "min_p", "u"))
    k = s["top_k"].cpu().numpy()
    chance = np.empty(len(logits))
    for r, x in enumerate(logits):
        if not heat[r] > 0:
            chance[r] = 0.0
            continue
        # only finite logits can be drawn; by falling value, equal ones by index
        place = np.flatnonzero(x > -math.inf)
        place = place[np.lexsort((place, -x[place]))]
        if k[r] > 0:
            place = place[: k[r]]
        w = np.exp((x[place] - x[place[0]]) / heat[r])
        if p[r] < 1:
            share = np.concatenate(([0.0], np.cumsum(w)[:-1])) / w.sum()
            n = max(1, int(np.searchsorted(share, p[r], side="left")))
            place, w = place[:n], w[:n]
        sure = w >= m[r]
        place, w = place[sure], w[sure]
        by_index = np.argsort(place)
        place, w = place[by_index], w[by_index]
        at = min(int(np.searchsorted(np.cumsum(w), u[r] * w.sum(), side="right")), len(w) - 1)
        chance[r] = math.log(w[at]) - math.log(w.sum())
    return [None, torch.from_numpy(chance)]
