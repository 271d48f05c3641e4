"""Float64 statements of the serving operators (the definitions in include/moe_serving.h).

Plain loops over sequences, heads and pages in numpy; nothing here is shared with the CUDA
library.  The cache append's rounding rules are defined on float32 values, so it is stated with
single float32 operations and is exact; attention and the linear product are float64 with an
error bound beside the value; draft verification is whole numbers.
"""
from __future__ import annotations

import math

import numpy as np

E4M3 = np.array([(-1.0 if b & 128 else 1.0) *
                 (math.nan if (b & 127) == 127 else
                  (b & 7) * 2.0 ** -9 if (b >> 3 & 15) == 0 else
                  (1 + (b & 7) / 8) * 2.0 ** ((b >> 3 & 15) - 7)) for b in range(256)])
_POS = E4M3[:127]                                   # ascending, 0 .. 448


def e4m3_encode(v: np.ndarray) -> np.ndarray:
    """Nearest E4M3 code, ties to the even code, saturating at 448; NaN -> 0x7F."""
    a = np.abs(np.asarray(v, np.float64))
    mid = (_POS[1:] + _POS[:-1]) / 2
    lo = np.searchsorted(mid, a, side="left")       # a <= mid[lo]
    tie = (lo < 126) & (a == mid[np.minimum(lo, 125)]) & (lo % 2 == 1)
    code = np.where(tie, lo + 1, lo).astype(np.uint8)
    code = code | (np.signbit(v).astype(np.uint8) << 7)
    return np.where(np.isnan(v), np.uint8(0x7F), code)


def scale_exponent(a: float) -> int:
    """Least e in [-64, 119] with a <= 448 * 2^e."""
    e = -64
    while e < 119 and a > 448.0 * 2.0 ** e:
        e += 1
    return e


def rotate(x, cos, sin, interleaved: bool):
    """x float32 [..., D]; cos, sin float32 [..., r/2] for the same rows; single f32 operations."""
    x = x.astype(np.float32).copy()
    half = cos.shape[-1]
    lo = np.arange(0, 2 * half, 2) if interleaved else np.arange(half)
    hi = lo + 1 if interleaved else lo + half
    a, b = x[..., lo], x[..., hi]
    x[..., lo] = a * cos - b * sin
    x[..., hi] = b * cos + a * sin
    return x


def kv_append(codes, scales, values, q_offsets, seq_lens, page_table):
    """Append one plane's values float32 [T, heads, D] (K's already rotated); codes uint8
    [pages, heads, P, D] and scales float32 [pages, heads] are changed in place."""
    num_pages, heads, P, _ = codes.shape
    for b in range(len(seq_lens)):
        r0, r1 = int(q_offsets[b]), int(q_offsets[b + 1])
        start = int(seq_lens[b]) - (r1 - r0)
        places = [i for i in range(max(start, 0), min(int(seq_lens[b]), page_table.shape[1] * P))]
        for pi in sorted({i // P for i in places}):
            page = int(page_table[b, pi])
            if not 0 <= page < num_pages:
                continue
            here = [i for i in places if i // P == pi]
            first = here[0] % P
            for h in range(heads):
                new = np.stack([values[r0 + i - start, h] for i in here])
                fresh = np.float32(2.0 ** scale_exponent(float(np.abs(new).max())))
                old = scales[page, h]
                s = fresh if first == 0 else np.float32(max(old, fresh))
                if first > 0 and s > old:
                    was = E4M3[codes[page, h, :first]].astype(np.float32)
                    codes[page, h, :first] = e4m3_encode(was * np.float32(old / s))
                for i, row in zip(here, new):
                    codes[page, h, i % P] = e4m3_encode((row / s).astype(np.float32))
                scales[page, h] = s


def attention(q, k_codes, k_scales, v_codes, v_scales, q_offsets, seq_lens, page_table, scale,
              window=0):
    """q float64 [T, hq, D].  Returns out [T, hq, D], lse [T, hq] and error bounds of both for a
    computation with f32 accumulation and the weights exp(s - max) * v_scale rounded to f16."""
    T, hq, D = q.shape
    num_pages, hkv, P, _ = k_codes.shape
    out, lse = np.zeros((T, hq, D)), np.full((T, hq), -np.inf)
    eo, el = np.zeros((T, hq, D)), np.zeros((T, hq))
    for b in range(len(seq_lens)):
        r0, r1 = int(q_offsets[b]), int(q_offsets[b + 1])
        n = int(seq_lens[b])
        start = n - (r1 - r0)
        js = np.arange(max(0, min(n, page_table.shape[1] * P)))
        pages = page_table[b, js // P].astype(np.int64) if js.size else js
        good = (pages >= 0) & (pages < num_pages)
        js, pages = js[good], pages[good]
        for h in range(hkv):
            K = E4M3[k_codes[pages, h, js % P]]
            V = E4M3[v_codes[pages, h, js % P]]
            ks, vs = k_scales[pages, h].astype(np.float64), v_scales[pages, h].astype(np.float64)
            for t in range(r0, r1):
                at = start + t - r0
                see = js <= at
                if window:
                    see &= js > at - window
                if not see.any():
                    continue
                k, v, a, c = K[see], V[see], ks[see], vs[see]
                for r in range(h * hq // hkv, (h + 1) * hq // hkv):
                    s = (k @ q[t, r]) * a * scale
                    m = s.max()
                    p = np.exp(s - m)
                    l = p.sum()
                    out[t, r] = (p * c) @ v / l
                    lse[t, r] = m + np.log(l)
                    # relative error of a weight: the score's f32 accumulation (two roundings,
                    # possibly truncations, per 16 products), its scaling, and exp
                    mag = (np.abs(k) @ np.abs(q[t, r])) * a * scale
                    rel = (D / 8 + 4) * 2.0 ** -23 * mag + 2.0 ** -22 * (np.abs(s) + abs(m)) + 2.0 ** -20
                    w = p * c
                    f16 = np.maximum(2.0 ** -11 * w, 2.0 ** -25 * w.max())
                    eo[t, r] = ((w * rel + f16) @ np.abs(v)) / l + np.abs(out[t, r]) * (p @ rel / l) \
                        + (w @ np.abs(v)) / l * 2.0 ** -22 * (8 + math.log2(len(s)))
                    el[t, r] = p @ rel / l + 2.0 ** -21 + abs(lse[t, r]) * 2.0 ** -22
    return out, lse, eo, el


def linear(x, w):
    """x float64 [T, K], w float64 [N, K]: y and the bound of an f32 accumulation in any order
    of groups of 16 products (two roundings, possibly truncations, per group)."""
    y, mag = x @ w.T, np.abs(x) @ np.abs(w).T
    return y, mag * (x.shape[1] / 8 + 16) * 2.0 ** -23


def verify_draft(draft_ids, n_draft, target, draft, u_accept, u_sample):
    """Python integers throughout; target [B, n+1, V] and draft [B, n, V] or None, float32."""
    B, n = draft_ids.shape
    V = target.shape[2]
    ids = np.full((B, n + 1), -1, np.int32)
    counts = np.zeros(B, np.int32)

    def masses(w):
        w = np.clip(np.where(np.isnan(w), np.float32(0), w.astype(np.float32)), 0, 1)
        return [int(x) for x in np.floor(w.astype(np.float64) * 2.0 ** 40)]

    for b in range(B):
        m = int(n_draft[b]) if n_draft is not None else n
        c = 0
        while c < m:
            x = int(draft_ids[b, c])
            if not 0 <= x < V:
                break
            qx = np.float32(draft[b, c, x]) if draft is not None else np.float32(1)
            if not np.float32(u_accept[b, c]) * qx < np.float32(target[b, c, x]):
                break
            ids[b, c] = x
            c += 1
        p = target[b, c].astype(np.float32)
        w = p.copy()
        if c < m:
            if draft is not None:
                w = w - draft[b, c].astype(np.float32)
            elif 0 <= int(draft_ids[b, c]) < V:
                w[int(draft_ids[b, c])] -= np.float32(1)
        mass = masses(w)
        if sum(mass) == 0:
            mass = masses(p)
        total = sum(mass)
        counts[b] = c
        if total:
            u = np.float32(min(max(float(u_sample[b]), 0.0), 1.0))
            goal = (min(int(float(u) * 2 ** 24), 2 ** 24 - 1) * total) >> 24
            run = 0
            for v, x in enumerate(mass):
                run += x
                if run > goal:
                    ids[b, c] = v
                    break
    return ids, counts
