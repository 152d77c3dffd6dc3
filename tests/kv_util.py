"""Helpers of the key-value cache tests: random caches on the host and their
device copies."""

import numpy as np
import torch

import dequant_gemv_rht_amd as dq
import workloads as W
from oracle import kvcache as OK

from gpu_util import dev, dev_u32


def sign_words(heads, d, rng):
    return W.sign_bits(heads * d, rng)


def random_cache(rng, pages, page, heads, d, bits, rotated=False, channel_scale=None):
    """(host arrays dict, KVCache): normal rows, coded by the oracle's rule."""
    host = {"signs": sign_words(heads, d, rng) if rotated else None}
    for which in "kv":
        x = rng.standard_normal((pages, heads, page, d)).astype(np.float32)
        if channel_scale is not None:
            x *= np.asarray(channel_scale, np.float32)
        if bits == 16:
            host[which + "_params"] = None
            host[which] = OK.pack_pages(which, x.astype(np.float16), 16)
        else:
            q, s, z = OK.code_rows(x, bits)
            host[which + "_params"] = np.stack([s, z], -1)
            host[which] = OK.pack_pages(which, q, bits)
    return host, device_cache(host, page, heads, d, bits)


def device_cache(host, page, heads, d, bits):
    t = {n: None if host[n] is None else dev(host[n]) for n in ("k", "v", "k_params", "v_params")}
    signs = None if host["signs"] is None else dev_u32(host["signs"])
    return dq.KVCache(bits, d, heads, page, t["k"], t["v"], t["k_params"], t["v_params"], signs)


def values(host, which, bits, d, page):
    return OK.dequant_pages(which, host[which], host[which + "_params"], bits, d, page)


def guarded(rows, cols, ld, fill=float("nan")):
    """A view [rows][cols] of row stride ld, and the whole buffer, filled with `fill`."""
    buf = torch.full((rows + 2, ld), fill, dtype=torch.float16, device="cuda")
    return buf[1:rows + 1, :cols], buf
