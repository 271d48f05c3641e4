"""Inputs and host copies for the serving operators' tests."""
from __future__ import annotations

import numpy as np
import torch

import nvfp4_grouped_gemm_gb300 as moe

DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


def activations(rng, shape, dtype, amp=1.0):
    return torch.from_numpy((rng.standard_normal(shape) * amp).astype(np.float32)).to(DT[dtype])


class Batch:
    """Sequences as (cached, new) token counts with a page table over shuffled pages; the table's
    unused entries are out of range and the spare pages are shared by nobody."""

    def __init__(self, rng, pairs, page, spare=2, extra_cols=1):
        self.pairs, self.page = pairs, page
        lens = [p + n for p, n in pairs]
        counts = [max(0, -(-v // page)) for v in lens]
        self.num_pages = sum(counts) + spare
        order = rng.permutation(self.num_pages)
        self.table = np.full((len(pairs), max(counts + [1]) + extra_cols), -7, np.int32)
        at = 0
        for b, c in enumerate(counts):
            self.table[b, :c] = order[at:at + c]
            at += c
        self.lens = np.array(lens, np.int32)
        self.offsets = np.array([0] + list(np.cumsum([n for _, n in pairs])), np.int32)
        self.T = int(self.offsets[-1])

    def device(self):
        return moe.SeqBatch(torch.from_numpy(self.offsets).cuda(), torch.from_numpy(self.lens).cuda(),
                            torch.from_numpy(self.table).cuda())


def cache_planes(rng, num_pages, heads, page, dim, nan_fill=False):
    """Host planes: codes uint8, scales powers of two."""
    def codes():
        c = rng.integers(0, 127, size=(num_pages, heads, page, dim), dtype=np.uint8)
        return c | (rng.integers(0, 2, size=c.shape, dtype=np.uint8) << 7)
    def scales():
        return (2.0 ** rng.integers(-9, -5, size=(num_pages, heads))).astype(np.float32)
    return codes(), scales(), codes(), scales()


def device_cache(planes):
    kc, ks, vc, vs = (torch.from_numpy(p.copy()).cuda() for p in planes)
    return moe.PagedKvCache(kc, vc, ks, vs)


def zeros_ws(nbytes):
    assert nbytes > 0
    return torch.zeros(nbytes, dtype=torch.uint8, device="cuda")
