"""The serving operators around the MoE layer, as workloads: appending keys and values to the
paged 8-bit cache with the rotary rotation, attention over that cache, the NVFP4
matrix-vector product, and the verification of drafted tokens.

``listed()`` names the workloads, ``draw(rng)`` gives more of the same ranges, ``prepare``
makes a workload's inputs on the GPU, ``run`` makes one pass through its operator (in plain
torch operations, or with ``own`` set through the library's calls), ``exact`` gives the same
outputs from the definitions in 64 bits, and ``work`` counts the bytes and operations a pass
cannot do without.
"""
import math

import torch

own = False

_DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


# ---------------------------------------------------------------------------
# workloads
# ---------------------------------------------------------------------------
def listed():
    return [
        # one new token of one sequence: a decode step's append, where only latency counts
        {"name": "append_token", "op": "append", "B": 1, "n": 1, "ragged": False, "past_lo": 1000,
         "past_hi": 1000, "q_heads": 32, "kv_heads": 8, "D": 128, "page": 64, "rotary": 128,
         "interleaved": False, "dtype": "bf16"},
        # six prompts of different lengths entering the cache together (about 4000 tokens)
        {"name": "append_prompts", "op": "append", "B": 6, "n": 2048, "ragged": True, "past_lo": 0,
         "past_hi": 300, "q_heads": 32, "kv_heads": 8, "D": 128, "page": 64, "rotary": 128,
         "interleaved": True, "dtype": "f16"},
        # one sequence's decode step over a long context
        {"name": "attention_token", "op": "attention", "B": 1, "n": 1, "ragged": False,
         "past_lo": 32766, "past_hi": 32766, "q_heads": 64, "kv_heads": 8, "D": 128, "page": 64,
         "window": 0, "dtype": "bf16"},
        # a serving batch's decode step: 64 sequences of very different lengths
        {"name": "attention_batch", "op": "attention", "B": 64, "n": 1, "ragged": False,
         "past_lo": 100, "past_hi": 16000, "q_heads": 32, "kv_heads": 8, "D": 128, "page": 64,
         "window": 0, "dtype": "bf16"},
        # drafted tokens of 16 sequences scored together (a verify batch of 128 tokens), five
        # query heads per key head, small heads and small pages
        {"name": "attention_verify", "op": "attention", "B": 16, "n": 8, "ragged": False,
         "past_lo": 500, "past_hi": 9000, "q_heads": 40, "kv_heads": 8, "D": 64, "page": 16,
         "window": 0, "dtype": "f16"},
        # a chunk of a long prompt after 6144 cached tokens
        {"name": "attention_prompt", "op": "attention", "B": 1, "n": 2048, "ragged": False,
         "past_lo": 6144, "past_hi": 6144, "q_heads": 32, "kv_heads": 8, "D": 128, "page": 64,
         "window": 0, "dtype": "bf16"},
        # the q/k/v projection of one token at the decode layer's hidden size
        {"name": "linear_token", "op": "linear", "T": 1, "K": 2560, "N": 5120, "dtype": "bf16",
         "out": "bf16"},
        # a small projection of a few tokens with an odd number of rows
        {"name": "linear_odd", "op": "linear", "T": 5, "K": 640, "N": 2561, "dtype": "bf16",
         "out": "f32"},
        # the language-model head for a verify batch of 16 tokens
        {"name": "linear_head", "op": "linear", "T": 16, "K": 4096, "N": 131101, "dtype": "bf16",
         "out": "f32"},
        # four drafted tokens of one sequence
        {"name": "verify_one", "op": "verify", "B": 1, "n": 4, "V": 32003, "dtype": "f32",
         "draft_probs": True},
        # eight drafted tokens of each of 64 sequences at a large vocabulary
        {"name": "verify_batch", "op": "verify", "B": 64, "n": 8, "V": 151937, "dtype": "f32",
         "draft_probs": True},
        # drafts looked up in the text (no draft distribution), half-precision probabilities
        {"name": "verify_lookup", "op": "verify", "B": 16, "n": 3, "V": 100003, "dtype": "bf16",
         "draft_probs": False},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["append", "attention", "attention", "linear", "verify"])
    if op == "append":
        B = _log_int(rng, 1, 96)
        n = _log_int(rng, 1, max(1, 4096 // B))
        D = rng.choice([64, 128, 128, 256])
        past = _log_int(rng, 1, 4000)
        return {"op": op, "B": B, "n": n, "ragged": rng.random() < 0.5, "past_lo": past // 3,
                "past_hi": past, "q_heads": rng.choice([1, 2, 4, 5, 8]) * 4, "kv_heads": 4, "D": D,
                "page": rng.choice([16, 32, 64, 128]), "rotary": rng.choice([D, D, D // 2]),
                "interleaved": rng.random() < 0.5, "dtype": rng.choice(["bf16", "f16"])}
    if op == "attention":
        D = rng.choice([64, 128, 128, 256])
        kv = rng.choice([1, 2, 4, 8])
        group = rng.choice([1, 2, 4, 5, 7, 8, 12, 16])
        page = rng.choice([16, 32, 64, 128])
        window = rng.choice([0, 0, 0, 777])
        dtype = rng.choice(["bf16", "f16"])
        if rng.random() < 0.25:           # a chunk of a prompt
            n = _log_int(rng, 64, 1500)
            return {"op": op, "B": rng.randint(1, 3), "n": n, "ragged": rng.random() < 0.5,
                    "past_lo": 0, "past_hi": _log_int(rng, 1, 1500), "q_heads": kv * min(group, 4),
                    "kv_heads": kv, "D": min(D, 128), "page": page, "window": window,
                    "dtype": dtype}
        B = _log_int(rng, 1, 96)
        past = _log_int(rng, 1, min(60000, 400000 // B))
        return {"op": op, "B": B, "n": _log_int(rng, 1, 8), "ragged": rng.random() < 0.5,
                "past_lo": max(0, past // rng.choice([1, 8, 64])), "past_hi": past,
                "q_heads": kv * group, "kv_heads": kv, "D": D, "page": page, "window": window,
                "dtype": dtype}
    if op == "linear":
        K = 32 * _log_int(rng, 2, 200)
        K = 3104 if K == 3072 else K
        N = _log_int(rng, 64, 100000)
        N = 3073 if N == 3072 else N
        return {"op": op, "T": _log_int(rng, 1, 32), "K": K, "N": N,
                "dtype": rng.choice(["bf16", "f16"]), "out": rng.choice(["f32", "bf16", "f16"])}
    return {"op": op, "B": _log_int(rng, 1, 64), "n": rng.randint(1, 8),
            "V": _log_int(rng, 200, 150000), "dtype": rng.choice(["f32", "bf16", "f16"]),
            "draft_probs": rng.random() < 0.7}


def _spaced(lo, hi, count):
    """`count` whole numbers from lo to hi, evenly spaced in their logarithm."""
    if count == 1:
        return [hi]
    a, b = math.log(lo + 1), math.log(hi + 1)
    return [int(round(math.exp(a + (b - a) * i / (count - 1)))) - 1 for i in range(count)]


def _lengths(case):
    """(cached tokens before the call, new tokens) of each sequence, in no order that matters."""
    past = _spaced(case["past_lo"], case["past_hi"], case["B"])
    new = [max(1, v) for v in _spaced(max(1, case["n"] // 8), case["n"], case["B"])] \
        if case["ragged"] else [case["n"]] * case["B"]
    return list(zip(past, reversed(new)))


def work(case):
    if case["op"] in ("append", "attention"):
        pairs, D, hq, hkv, page = (_lengths(case), case["D"], case["q_heads"], case["kv_heads"],
                                   case["page"])
        T = sum(n for _, n in pairs)
    if case["op"] == "append":
        b = T * D * (2 * (2 * hq + 2 * hkv) + 2 * hkv) + T * case["rotary"] * 4 + T * 4
        touched = sum((p + n - 1) // page - p // page + 1 for p, n in pairs)
        return {"bytes": b + touched * hkv * 8, "flops": 3 * T * case["rotary"] * (hq + hkv)}
    if case["op"] == "attention":
        w = case["window"]
        seen = keys = 0
        for p, n in pairs:
            seen += sum(min(p + i + 1, w) if w else p + i + 1 for i in range(n))
            keys += min(p + n, w + n - 1) if w else p + n
        pages = keys / page
        return {"bytes": keys * hkv * D * 2 + pages * (hkv * 8 + 4) + T * hq * (D * 4 + 4),
                "flops": 4 * D * hq * seen}
    if case["op"] == "linear":
        T, K, N = case["T"], case["K"], case["N"]
        out = 4 if case["out"] == "f32" else 2
        return {"bytes": N * K // 2 + N * K // 16 + T * K * 2 + T * N * out, "flops": 2 * T * N * K}
    # the target row that the last token comes from, and the draft row beside it where a
    # draft was refused (about half of the sequences), of each sequence
    size = 4 if case["dtype"] == "f32" else 2
    rows = case["B"] * (1.5 if case["draft_probs"] else 1)
    return {"bytes": rows * case["V"] * size, "flops": rows * case["V"] * 2}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _i32(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _batch(case, g, spare=3):
    """Ragged batch: offsets of the new tokens, lengths, and a page table over shuffled pages."""
    pairs = _lengths(case)
    order = torch.randperm(len(pairs), generator=g, device="cuda").tolist()
    pairs = [pairs[i] for i in order]
    page = case["page"]
    lens = [p + n for p, n in pairs]
    counts = [(v + page - 1) // page for v in lens]
    num_pages, cols = sum(counts) + spare, max(counts)
    perm = torch.randperm(num_pages, generator=g, device="cuda").to(torch.int32)
    first = torch.tensor([0] + counts[:-1], device="cuda").cumsum(0)
    col = torch.arange(cols, device="cuda")
    used = col[None, :] < torch.tensor(counts, device="cuda")[:, None]
    table = torch.where(used, perm[(first[:, None] + col[None, :]).clamp(max=num_pages - 1)], 0)
    offsets = [0]
    for _, n in pairs:
        offsets.append(offsets[-1] + n)
    return {"q_offsets": _i32(offsets), "seq_lens": _i32(lens),
            "page_table": table.to(torch.int32).contiguous(), "num_pages": num_pages,
            "T": offsets[-1], "max_n": max(n for _, n in pairs), "max_len": max(lens)}


def _cache(case, g, num_pages):
    """E4M3 codes with the spread of unit-variance keys and values, and power-of-two scales of
    each page and head (some heads twice or four times louder than others)."""
    shape = (num_pages, case["kv_heads"], case["page"], case["D"])
    out = []
    for _ in range(2):
        codes = torch.empty(shape, dtype=torch.uint8, device="cuda")
        for part in codes.split(max(1, (1 << 27) // codes[0].numel())):
            part.copy_((torch.randn(part.shape, generator=g, device="cuda") * 90)
                       .clamp_(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8))
        scales = torch.exp2(torch.randint(-8, -5, shape[:2], generator=g, device="cuda").float())
        out += [codes, scales]
    return {"k_codes": out[0], "k_scales": out[1], "v_codes": out[2], "v_scales": out[3]}


def _heads(g, T, heads, D, dtype):
    return torch.randn(T, heads, D, generator=g, device="cuda").to(dtype)


def prepare(case, seed):
    g = _gen(seed)
    s = {"case": case}
    if case["op"] in ("append", "attention"):
        s.update(_batch(case, g))
        s.update(_cache(case, g, s["num_pages"]))
        dt = _DT[case["dtype"]]
        s["q"] = _heads(g, s["T"], case["q_heads"], case["D"], dt)
        s["out"] = torch.empty_like(s["q"])
    if case["op"] == "append":
        s["k"] = _heads(g, s["T"], case["kv_heads"], case["D"], dt)
        s["v"] = _heads(g, s["T"], case["kv_heads"], case["D"], dt)
        rot = case["rotary"]
        inv = 10000.0 ** (-torch.arange(0, rot, 2, device="cuda", dtype=torch.float64) / rot)
        angle = torch.arange(s["max_len"], device="cuda", dtype=torch.float64)[:, None] * inv
        s["cos"], s["sin"] = angle.cos().float(), angle.sin().float()
    elif case["op"] == "attention":
        # slots past a sequence's end hold whatever was there: here NaN codes
        page = case["page"]
        b = torch.arange(case["B"], device="cuda")
        last = s["page_table"][b, ((s["seq_lens"] - 1) // page).long()].long()
        stale = torch.arange(page, device="cuda") >= ((s["seq_lens"] - 1) % page + 1)[:, None]
        for plane in ("k_codes", "v_codes"):
            pages = s[plane][last]
            pages.masked_fill_(stale[:, None, :, None], 0x7F)
            s[plane][last] = pages
        s["scale"] = case["D"] ** -0.5
        s["lse"] = torch.empty(s["T"], case["q_heads"], device="cuda")
    elif case["op"] == "linear":
        N, K = case["N"], case["K"]
        s["codes"] = torch.randint(0, 256, (1, N, K // 2), generator=g, device="cuda",
                                   dtype=torch.uint8)
        s["scales"] = torch.randint(0x08, 0x31, (1, N, K // 16), generator=g, device="cuda",
                                    dtype=torch.uint8)
        s["x"] = torch.randn(case["T"], K, generator=g, device="cuda").to(_DT[case["dtype"]])
        s["y"] = torch.empty(case["T"], N, device="cuda", dtype=_DT[case["out"]])
    else:
        B, n, V, dt = case["B"], case["n"], case["V"], _DT[case["dtype"]]
        logits = torch.randn(B, n + 1, V, generator=g, device="cuda") * 3
        s["target_probs"] = torch.softmax(logits, -1).to(dt)
        near = torch.softmax(logits[:, :n] + torch.randn(B, n, V, generator=g, device="cuda") * 0.6,
                             -1)
        s["draft_ids"] = torch.multinomial(near.view(B * n, V), 1, generator=g) \
            .view(B, n).to(torch.int32)
        s["draft_probs"] = near.to(dt) if case["draft_probs"] else None
        s["n_draft"] = torch.randint(max(0, n - 1), n + 1, (B,), generator=g, device="cuda",
                                     dtype=torch.int32)
        s["u_accept"] = torch.rand(B, n, generator=g, device="cuda")
        s["u_sample"] = torch.rand(B, generator=g, device="cuda")
        s["out_ids"] = torch.empty(B, n + 1, dtype=torch.int32, device="cuda")
        s["n_accepted"] = torch.empty(B, dtype=torch.int32, device="cuda")
    if own:
        _prepare_own(s)
    return s


def _prepare_own(s):
    """The handles and workspaces that a serving loop keeps."""
    import nvfp4_grouped_gemm_gb300 as moe
    case, op = s["case"], s["case"]["op"]
    if op in ("append", "attention"):
        s["cache"] = moe.PagedKvCache(s["k_codes"], s["v_codes"], s["k_scales"], s["v_scales"])
        s["batch"] = moe.SeqBatch(s["q_offsets"], s["seq_lens"], s["page_table"])
    if op == "append":
        n = moe.kv_append_workspace_bytes()
    elif op == "attention":
        n = moe.attention_workspace_bytes(case["q_heads"], case["kv_heads"], case["D"])
    elif op == "linear":
        s["bank"] = moe.NvFp4Bank(s["codes"], s["scales"])
        n = moe.linear_workspace_bytes(case["T"], case["N"], case["K"])
    else:
        n = moe.verify_workspace_bytes(case["B"], case["V"])
    s["ws"] = torch.zeros(n, dtype=torch.uint8, device="cuda")
    s["moe"] = moe


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------
def run(state):
    op = state["case"]["op"]
    if own:
        return _OWN[op](state)
    return _PLAIN[op](state)


def _append_own(s):
    s["moe"].moe_kv_append_rope_e4m3(s["cache"], s["batch"], s["k"], s["v"], s["cos"], s["sin"],
                                     s["ws"], q=s["q"], q_out=s["out"],
                                     interleaved=s["case"]["interleaved"])
    return _append_outputs(s)


def _append_outputs(s):
    f8 = torch.float8_e4m3fn
    return {"q": s["out"], "k": s["k_codes"].view(f8), "k_scales": s["k_scales"],
            "v": s["v_codes"].view(f8), "v_scales": s["v_scales"]}


def _attention_own(s):
    s["moe"].moe_attention_paged_e4m3(s["q"], s["cache"], s["batch"], s["out"], s["ws"],
                                      scale=s["scale"], window=s["case"]["window"], lse=s["lse"])
    return {"out": s["out"], "lse": s["lse"]}


def _linear_own(s):
    s["moe"].moe_linear_nvfp4(s["x"], s["bank"], s["y"], s["ws"])
    return s["y"]


def _verify_own(s):
    s["moe"].moe_verify_draft(s["draft_ids"], s["target_probs"], s["u_accept"], s["u_sample"],
                              s["out_ids"], s["n_accepted"], s["ws"],
                              draft_probs=s["draft_probs"], n_draft=s["n_draft"])
    return {"ids": s["out_ids"], "n_accepted": s["n_accepted"]}


_OWN = {"append": _append_own, "attention": _attention_own, "linear": _linear_own,
        "verify": _verify_own}


# ---- plain forms ----------------------------------------------------------
def _slots(s):
    """For each new token: its sequence, its place in the sequence, its page and slot."""
    t = torch.arange(s["T"], device="cuda")
    off = s["q_offsets"].long()
    b = torch.searchsorted(off[1:].contiguous(), t, right=True)
    place = s["seq_lens"].long()[b] - off[b + 1] + t
    page = s["case"]["page"]
    return b, place, s["page_table"][b, place // page].long(), place % page


def _rotate(x, cos, sin, interleaved):
    """x [T, heads, D] in 32 bits; the first 2 * cos.shape[1] values of each head are rotated."""
    half = cos.shape[1]
    c, n = cos[:, None, :], sin[:, None, :]
    rot, rest = x[..., :2 * half], x[..., 2 * half:]
    if interleaved:
        a, b = rot[..., 0::2], rot[..., 1::2]
        rot = torch.stack((a * c - b * n, b * c + a * n), -1).flatten(-2)
    else:
        a, b = rot[..., :half], rot[..., half:]
        rot = torch.cat((a * c - b * n, b * c + a * n), -1)
    return torch.cat((rot, rest), -1)


def _append_plane(codes, scales, values, pages, slots):
    """Write `values` [T, heads, D] at (pages, slots): each touched page's scale is the least
    power of two that holds its new values, or its old scale if that is larger and the page
    had tokens before; codes written earlier follow a scale that grew."""
    f8 = torch.float8_e4m3fn
    touched, at = torch.unique(pages, return_inverse=True)
    count = touched.numel()
    heads = values.shape[1]
    peak = torch.zeros(count, heads, device="cuda").scatter_reduce_(
        0, at[:, None].expand(-1, heads), values.abs().amax(-1), "amax")
    first = torch.full((count,), 1 << 30, device="cuda", dtype=torch.long).scatter_reduce_(
        0, at, slots, "amin")
    m, e = torch.frexp(peak)
    e = torch.where(m <= 0.875, e - 9, e - 8).clamp(-64, 119)
    e = torch.where(peak > 0, e, torch.full_like(e, -64))
    fresh = torch.ldexp(torch.ones_like(peak), e)
    old = scales[touched]
    new = torch.where((first > 0)[:, None], torch.maximum(old, fresh), fresh)
    earlier = torch.arange(codes.shape[2], device="cuda")[None, :] < first[:, None]
    had = codes[touched]
    moved = (had.view(f8).float() * (old / new)[:, :, None, None]).to(f8).view(torch.uint8)
    grew = (new > old)[:, :, None, None] & earlier[:, None, :, None]
    codes[touched] = torch.where(grew, moved, had)
    scales[touched] = new
    codes[pages, :, slots] = (values / new[at][:, :, None]).to(f8).view(torch.uint8)


def _append_plain(s):
    case = s["case"]
    _, place, pages, slots = _slots(s)
    cos, sin = s["cos"][place], s["sin"][place]
    s["out"].copy_(_rotate(s["q"].float(), cos, sin, case["interleaved"]))
    _append_plane(s["k_codes"], s["k_scales"],
                  _rotate(s["k"].float(), cos, sin, case["interleaved"]), pages, slots)
    _append_plane(s["v_codes"], s["v_scales"], s["v"].float(), pages, slots)
    return _append_outputs(s)


def _gathered(s, codes, scales):
    """A plane as [B, heads, padded length, D] in 32 bits, through the page table."""
    table = s["page_table"].long()
    x = codes[table].view(torch.float8_e4m3fn).float() * scales[table][..., None, None]
    return x.transpose(1, 2).flatten(2, 3)


def _attention_plain(s):
    case = s["case"]
    hq, hkv, D = case["q_heads"], case["kv_heads"], case["D"]
    b, place, _, _ = _slots(s)
    B, n = case["B"], s["max_n"]
    i = torch.arange(s["T"], device="cuda") - s["q_offsets"].long()[b]
    q = torch.zeros(B, n, hq, D, device="cuda")
    q[b, i] = s["q"].float()
    q = q.view(B, n, hkv, hq // hkv, D).permute(0, 2, 3, 1, 4).flatten(2, 3)
    at = torch.full((B, n), -1, device="cuda", dtype=torch.long)
    at[b, i] = place
    k = _gathered(s, s["k_codes"], s["k_scales"])
    L = k.shape[2]
    scores = torch.matmul(q, k.transpose(-1, -2)).view(B, hkv, hq // hkv, n, L)
    del k
    j = torch.arange(L, device="cuda")
    sees = j <= at[..., None]
    if case["window"]:
        sees &= j > at[..., None] - case["window"]
    scores = torch.where(sees[:, None, None], scores * s["scale"], float("-inf"))
    top = scores.amax(-1, keepdim=True)
    p = torch.exp(scores - torch.where(top > float("-inf"), top, torch.zeros_like(top)))
    del scores
    total = p.sum(-1, keepdim=True)
    v = _gathered(s, s["v_codes"], s["v_scales"])
    v = torch.where((j < s["seq_lens"][:, None])[:, None, :, None], v, 0)
    o = torch.matmul(p.flatten(2, 3), v).view(B, hkv, hq // hkv, n, D)
    o = torch.where(total > 0, o / total, torch.zeros_like(o))
    lse = (top + total.log()).squeeze(-1).permute(0, 3, 1, 2).flatten(2)
    s["out"].copy_(o.permute(0, 3, 1, 2, 4).flatten(2, 3)[b, i])
    s["lse"].copy_(lse[b, i])
    return {"out": s["out"], "lse": s["lse"]}


_E2M1 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]


def _linear_plain(s):
    table = torch.tensor(_E2M1 + [-v for v in _E2M1], device="cuda")
    codes = s["codes"][0]
    w = torch.stack((table[(codes & 15).int()], table[(codes >> 4).int()]), -1).flatten(1)
    scale = s["scales"][0].view(torch.float8_e4m3fn).float()
    w = (w.view(w.shape[0], -1, 16) * scale[:, :, None]).flatten(1)
    s["y"].copy_(torch.matmul(s["x"].float(), w.t()))
    return s["y"]


def _mass(w):
    """Probabilities as whole numbers of 2^-40."""
    return (w.clamp(0, 1) * float(1 << 40)).to(torch.int64)


def _verify_plain(s):
    B, n = s["draft_ids"].shape
    ids = s["draft_ids"].long()
    target, drafts = s["target_probs"], s["draft_probs"]
    p = torch.gather(target[:, :n], 2, ids[..., None]).squeeze(-1).float()
    q = torch.gather(drafts, 2, ids[..., None]).squeeze(-1).float() if drafts is not None \
        else torch.ones_like(p)
    place = torch.arange(n, device="cuda")
    ok = (s["u_accept"] * q < p) & (place < s["n_draft"][:, None])
    count = ok.int().cumprod(1).sum(1)
    b = torch.arange(B, device="cuda")
    refused = count < s["n_draft"]
    at = count.clamp(max=n - 1)
    row = target[b, count].float()
    if drafts is not None:
        less = drafts[b, at].float()
    else:
        less = torch.zeros_like(row)
        less[b, ids[b, at]] = 1.0
    whole = _mass(row)
    mass = torch.where(refused[:, None], _mass(row - less), whole)
    mass = torch.where(mass.sum(1, keepdim=True) > 0, mass, whole)
    total = mass.sum(1)
    u = (s["u_sample"] * float(1 << 24)).floor().to(torch.int64)
    goal = u * (total >> 24) + ((u * (total & 0xFFFFFF)) >> 24)
    token = (mass.cumsum(1) <= goal[:, None]).sum(1)
    out = torch.where(place < count[:, None], ids, torch.full_like(ids, -1))
    out = torch.cat((out, torch.full_like(out[:, :1], -1)), 1)
    out[b, count] = token
    s["out_ids"].copy_(out)
    s["n_accepted"].copy_(count)
    return {"ids": s["out_ids"], "n_accepted": s["n_accepted"]}


_PLAIN = {"append": _append_plain, "attention": _attention_plain, "linear": _linear_plain,
          "verify": _verify_plain}


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------
def exact(case, seed):
    global own
    if case["op"] == "verify":            # whole numbers only
        return None
    was, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = was
    return {"append": _append_exact, "attention": _attention_exact, "linear": _linear_exact}[
        case["op"]](case, s)


def _e4m3_table():
    bytes_ = torch.arange(256, dtype=torch.uint8, device="cuda")
    return bytes_.view(torch.float8_e4m3fn).double()


def _append_exact(case, s):
    page, D, half = case["page"], case["D"], case["rotary"] // 2
    off, lens = s["q_offsets"].tolist(), s["seq_lens"].tolist()
    grid = _e4m3_table()
    planes = {"k": (grid[s["k_codes"].long()], s["k_scales"].double()),
              "v": (grid[s["v_codes"].long()], s["v_scales"].double())}
    if case["interleaved"]:
        low, high = torch.arange(0, 2 * half, 2), torch.arange(1, 2 * half, 2)
    else:
        low, high = torch.arange(half), torch.arange(half, 2 * half)

    def turned(x, place):
        x = x.double()
        y = x.clone()
        c, n = s["cos"][place].double()[:, None], s["sin"][place].double()[:, None]
        y[..., low] = x[..., low] * c - x[..., high] * n
        y[..., high] = x[..., low] * n + x[..., high] * c
        return y

    def near(x):
        """Nearest E4M3 value, ties to the even code."""
        a = x.abs().clamp(2.0 ** -60)
        step = torch.exp2(torch.floor(torch.log2(a)).clamp(min=-6) - 3)
        return torch.round(x / step) * step

    q = torch.empty(s["q"].shape, dtype=torch.float64, device="cuda")
    for b in range(case["B"]):
        lo, hi = off[b], off[b + 1]
        start = lens[b] - (hi - lo)
        place = torch.arange(start, lens[b], device="cuda")
        q[lo:hi] = turned(s["q"][lo:hi], place)
        new = {"k": turned(s["k"][lo:hi], place), "v": s["v"][lo:hi].double()}
        for at in range(start // page, (lens[b] - 1) // page + 1):
            a, z = max(start, at * page), min(lens[b], (at + 1) * page)
            number = int(s["page_table"][b, at])
            for name, (codes, scales) in planes.items():
                x = new[name][a - start:z - start].transpose(0, 1)          # [heads, tokens, D]
                need = torch.exp2(torch.ceil(torch.log2(x.abs().amax((1, 2)) / 448)).clamp(-64, 119))
                if a % page:
                    grown = torch.maximum(scales[number], need)
                    back = (scales[number] / grown)[:, None, None]
                    codes[number, :, :a % page] = near(codes[number, :, :a % page] * back)
                    need = grown
                scales[number] = need
                codes[number, :, a - at * page:z - at * page] = near(x / need[:, None, None])
    return {"q": q, "k": planes["k"][0], "k_scales": planes["k"][1], "v": planes["v"][0],
            "v_scales": planes["v"][1]}


def _attention_exact(case, s):
    hq, hkv, D, page, w = (case["q_heads"], case["kv_heads"], case["D"], case["page"],
                           case["window"])
    off, lens = s["q_offsets"].tolist(), s["seq_lens"].tolist()
    grid = _e4m3_table()
    group = hq // hkv
    out = torch.zeros(s["T"], hq, D, dtype=torch.float64, device="cuda")
    lse = torch.full((s["T"], hq), float("-inf"), dtype=torch.float64, device="cuda")
    for b in range(case["B"]):
        lo, hi, length = off[b], off[b + 1], lens[b]
        pages = s["page_table"][b, :(length + page - 1) // page].long()
        at = torch.arange(length - (hi - lo), length, device="cuda")[:, None]
        j = torch.arange(length, device="cuda")[None, :]
        hidden = (j > at) | ((j <= at - w) if w else torch.zeros_like(j, dtype=torch.bool))
        for h in range(hkv):
            k = (grid[s["k_codes"][pages, h].long()] * s["k_scales"][pages, h].double()
                 [:, None, None]).flatten(0, 1)[:length]
            v = (grid[s["v_codes"][pages, h].long()] * s["v_scales"][pages, h].double()
                 [:, None, None]).flatten(0, 1)[:length]
            for r in range(h * group, (h + 1) * group):
                score = (s["q"][lo:hi, r].double() @ k.t()) * s["scale"]
                score = score.masked_fill(hidden, float("-inf"))
                lse[lo:hi, r] = torch.logsumexp(score, 1)
                out[lo:hi, r] = torch.softmax(score, 1) @ v
    return {"out": out, "lse": lse}


def _linear_exact(case, s):
    values = _E2M1 + [-v for v in _E2M1]
    pair = torch.tensor([[values[c % 16], values[c // 16]] for c in range(256)],
                        dtype=torch.float64, device="cuda")
    grid = _e4m3_table()
    x = s["x"].double()
    y = torch.empty(case["T"], case["N"], dtype=torch.float64, device="cuda")
    for lo in range(0, case["N"], 16384):
        rows = slice(lo, min(case["N"], lo + 16384))
        w = pair[s["codes"][0, rows].long()].flatten(1)
        w = w * grid[s["scales"][0, rows].long()].repeat_interleave(16, 1)
        y[:, rows] = x @ w.t()
    return y
