"""Seeded caches and batches for the tests of the key/value cache."""
import numpy as np
import torch

import kv_ref
import ternary_weight_fwd_b200 as tw

DEV = "cuda"


def make_batch(new, lens, page, seed, behind=0, spare=2, width=None):
    """Page table (pages in a drawn order, unused entries -1), lengths and row starts, as numpy int32."""
    r = np.random.default_rng(seed)
    used = [-(-x // page) for x in lens]
    total = sum(used) + spare
    perm = r.permutation(total).astype(np.int32)
    table = np.full((len(lens), width or max(1, max(used))), -1, np.int32)
    at = 0
    for b, u in enumerate(used):
        table[b, :u] = perm[at:at + u]
        at += u
    q_start = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    return dict(table=table, lens=np.array(lens, np.int32), q_start=q_start, pages=total, rows=int(sum(new)) + behind,
                free=perm[at:])


def make_cache(pages, hk, page, d, seed, free=(), spread=0.3):
    """Codes and steps as numpy; the steps of pages that belong to nobody are NaN."""
    r = np.random.default_rng(seed)
    codes = [np.clip(np.rint(r.standard_normal((pages, hk, page, d)) * 40), -127, 127).astype(np.int8)
             for _ in range(2)]
    steps = [(0.02 * np.exp(spread * r.standard_normal((pages, hk)))).astype(np.float32) for _ in range(2)]
    for s in steps:
        s[list(free)] = np.nan
    return [codes[0], codes[1], steps[0], steps[1]]


def to_dev(cache):
    return tw.KVCache(*(torch.from_numpy(np.array(x)).to(DEV) for x in cache))


def dev(x):
    return torch.from_numpy(np.ascontiguousarray(x)).to(DEV)


def rows(shape, seed, dtype="bf16", scale=1.0):
    """(device tensor, the fp32 values it holds)."""
    x = (np.random.default_rng(seed).standard_normal(shape) * scale).astype(np.float32)
    if dtype == "bf16":
        x = kv_ref.bf16_round(x)
        return dev(x).to(torch.bfloat16), x
    return dev(x), x


def same_bits(a, b):
    return np.array_equal(np.ascontiguousarray(a).view(np.uint8), np.ascontiguousarray(b).view(np.uint8))
