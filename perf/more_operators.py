"""More operators around the paged 8-bit cache and the MoE layer, as workloads: attention for trees
of drafted tokens, the accumulated attention weight of cached tokens, eviction by that weight,
keeping a tree's accepted path, and the norms, gate and residual around a block.

``listed()`` names the workloads, ``draw(rng)`` gives more of the same ranges, ``prepare``
makes a workload's inputs on the GPU, ``run`` makes one pass through its operator (in plain
torch operations, or with ``own`` set through the library's calls), ``exact`` gives the same
outputs from the definitions in 64 bits, and ``work`` counts the bytes and operations a pass
cannot do without.
"""
import math
import random

import torch

own = False

_DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
_BYTES = {"bf16": 2, "f16": 2, "f32": 4}
_F8 = torch.float8_e4m3fn


# ---------------------------------------------------------------------------
# workloads
# ---------------------------------------------------------------------------
def listed():
    return [
        # a small tree of one sequence in a short chat: only latency counts
        {"name": "tree_small", "op": "tree", "B": 1, "n": 8, "ragged": False, "past_lo": 1000,
         "past_hi": 1000, "q_heads": 16, "kv_heads": 4, "D": 128, "page": 64, "window": 0,
         "dtype": "bf16"},
        # a serving batch's step: trees of up to 48 drafted tokens of 32 sequences
        {"name": "tree_batch", "op": "tree", "B": 32, "n": 48, "ragged": True, "past_lo": 500,
         "past_hi": 12000, "q_heads": 32, "kv_heads": 8, "D": 128, "page": 64, "window": 0,
         "dtype": "bf16"},
        # a layer with a sliding window, five query heads per key head, small heads and pages
        {"name": "tree_window", "op": "tree", "B": 5, "n": 37, "ragged": False, "past_lo": 300,
         "past_hi": 5000, "q_heads": 40, "kv_heads": 8, "D": 64, "page": 16, "window": 1001,
         "dtype": "f16"},
        # a decode step of one long sequence adds its attention to the running weights
        {"name": "weights_token", "op": "weights", "B": 1, "n": 1, "ragged": False,
         "past_lo": 32766, "past_hi": 32766, "q_heads": 64, "kv_heads": 8, "D": 128, "page": 64,
         "window": 0, "dtype": "bf16", "decay": 1.0},
        # the same for a serving batch of very different lengths, older steps fading
        {"name": "weights_batch", "op": "weights", "B": 64, "n": 1, "ragged": False,
         "past_lo": 100, "past_hi": 16000, "q_heads": 32, "kv_heads": 8, "D": 128, "page": 64,
         "window": 0, "dtype": "bf16", "decay": 0.984375},
        # prompts just read, judged by their last 32 tokens: the weights start here
        {"name": "weights_prompt", "op": "weights", "B": 6, "n": 32, "ragged": False,
         "past_lo": 1000, "past_hi": 16001, "q_heads": 40, "kv_heads": 8, "D": 64, "page": 16,
         "window": 0, "dtype": "f16", "decay": 0.0},
        # one sequence that has outgrown its budget by a few tokens
        {"name": "evict_one", "op": "evict", "B": 1, "len_lo": 1090, "len_hi": 1090,
         "budget": 1024, "ragged": False, "first": 4, "recent": 128, "kv_heads": 4, "D": 128,
         "page": 64},
        # long prompts of a serving batch cut down to a budget
        {"name": "evict_batch", "op": "evict", "B": 32, "len_lo": 2500, "len_hi": 16000,
         "budget": 4096, "ragged": True, "first": 0, "recent": 64, "kv_heads": 8, "D": 128,
         "page": 64},
        # the accepted path of one sequence's tree
        {"name": "keep_one", "op": "keep", "B": 1, "n": 16, "ragged": False, "past_lo": 2040,
         "past_hi": 2040, "kv_heads": 4, "D": 128, "page": 64},
        # accepted paths of a serving batch, small pages
        {"name": "keep_batch", "op": "keep", "B": 64, "n": 63, "ragged": True, "past_lo": 100,
         "past_hi": 3000, "kv_heads": 8, "D": 128, "page": 16},
        # one token between attention and the MoE layer
        {"name": "norm_token", "op": "norm", "T": 1, "H": 2560, "y": "bf16", "residual": "bf16",
         "normed": "bf16", "post": False, "pre": True, "gate": "none", "sigmoid": False,
         "scale": 1.0},
        # a prompt's tokens behind the MoE layer: norm of its output, gate of each token, next norm
        {"name": "norm_prompt", "op": "norm", "T": 4096, "H": 4096, "y": "f32", "residual": "bf16",
         "normed": "bf16", "post": True, "pre": True, "gate": "token", "sigmoid": True,
         "scale": 0.5},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["tree", "tree", "weights", "weights", "evict", "keep", "norm", "norm"])
    D = rng.choice([64, 128, 128, 256])
    kv = rng.choice([1, 2, 4, 8])
    group = rng.choice([1, 2, 4, 5, 7, 8])
    page = rng.choice([16, 32, 64, 128])
    if op == "tree":
        B, n = _log_int(rng, 1, 48), _log_int(rng, 1, 100)
        past = _log_int(rng, 1, max(2, min(40000, 300000 // B, 400000 * 32 // (B * n * group * kv))))
        return {"op": op, "B": B, "n": n, "ragged": rng.random() < 0.5,
                "past_lo": past // rng.choice([1, 8, 64]), "past_hi": past, "q_heads": kv * group,
                "kv_heads": kv, "D": D, "page": page, "window": rng.choice([0, 0, 0, 401, 30]),
                "dtype": rng.choice(["bf16", "f16"])}
    if op == "weights":
        B = _log_int(rng, 1, 96)
        n = _log_int(rng, 1, 64) if rng.random() < 0.5 else 1
        past = _log_int(rng, 1, max(2, min(60000, 400000 // B, 300000 * 32 // (B * n * group * kv))))
        return {"op": op, "B": B, "n": n, "ragged": rng.random() < 0.5,
                "past_lo": past // rng.choice([1, 8, 64]), "past_hi": past, "q_heads": kv * group,
                "kv_heads": kv, "D": D, "page": page, "window": rng.choice([0, 0, 0, 777]),
                "dtype": rng.choice(["bf16", "f16"]), "decay": rng.choice([1.0, 0.984375, 0.0])}
    if op == "evict":
        B = _log_int(rng, 1, 48)
        length = _log_int(rng, 20, min(60000, 120000 // B))
        budget = _log_int(rng, 4, max(5, length))
        return {"op": op, "B": B, "len_lo": max(1, length // rng.choice([1, 2, 6])),
                "len_hi": length, "budget": budget, "ragged": rng.random() < 0.5,
                "first": rng.choice([0, 1, 4]), "recent": rng.choice([0, 1, 33, 128]),
                "kv_heads": kv, "D": D, "page": page}
    if op == "keep":
        B = _log_int(rng, 1, 64)
        past = _log_int(rng, 1, 3000)
        return {"op": op, "B": B, "n": _log_int(rng, 1, 100), "ragged": rng.random() < 0.5,
                "past_lo": past // 3, "past_hi": past, "kv_heads": kv, "D": D, "page": page}
    T, H = _log_int(rng, 1, 4096), _log_int(rng, 64, 8192)
    H = H // 8 * 8 if rng.random() < 0.7 else H
    if H == 3072:
        H = 3080
    return {"op": op, "T": max(1, min(T, 9000000 // H)), "H": H, "y": rng.choice(["bf16", "f16", "f32"]),
            "residual": rng.choice(["bf16", "f16", "f32"]), "normed": rng.choice(["bf16", "f16"]),
            "post": rng.random() < 0.5, "pre": rng.random() < 0.9,
            "gate": rng.choice(["none", "token", "channel", "full"]), "sigmoid": rng.random() < 0.5,
            "scale": rng.choice([1.0, 0.5])}


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


def _evict_lengths(case):
    """(tokens, budget) of each sequence."""
    lens = _spaced(case["len_lo"], case["len_hi"], case["B"])
    low = max(1, case["budget"] // 2) if case["ragged"] else case["budget"]
    return list(zip(lens, _spaced(low, case["budget"], case["B"])))


def work(case):
    op = case["op"]
    if op == "norm":
        T, H = case["T"], case["H"]
        res, out = _BYTES[case["residual"]], _BYTES[case["normed"]] if case["pre"] else 0
        gate = {"none": 0, "token": T, "channel": H, "full": T * H}[case["gate"]] * 4
        b = T * H * (_BYTES[case["y"]] + 2 * res + out) + gate
        return {"bytes": b + 2 * H * (case["post"] + case["pre"]), "flops": 10 * T * H}
    D, page, hkv = case["D"], case["page"], case["kv_heads"]
    if op == "evict":
        lens = _evict_lengths(case)
        kept = sum(min(n, k) for n, k in lens)
        pages = sum(-(-min(n, k) // page) for n, k in lens)
        b = sum(n for n, _ in lens) * hkv * 4 + kept * hkv * (4 * D + 4 + 4) + pages * hkv * 16
        return {"bytes": b, "flops": kept * hkv * 2 * D}
    pairs = _lengths(case)
    if op == "keep":
        kept = sum(_kept_of(n) for _, n in pairs)
        return {"bytes": kept * hkv * 4 * D + kept * 4, "flops": kept * hkv * 2 * D}
    hq, w = case["q_heads"], case["window"]
    T = sum(n for _, n in pairs)
    seen = keys = 0
    for p, n in pairs:
        # a node of a tree sees its ancestors, about half as many as there are levels
        own_ = [1 + math.log2(i + 1) if op == "tree" else i + 1 for i in range(n)]
        seen += sum(min(p + v, w) if w else p + v for v in own_)
        keys += min(p + n, w + n - 1) if w else p + n
    pages = keys / page
    if op == "tree":
        return {"bytes": keys * hkv * D * 2 + pages * (hkv * 8 + 4) + T * hq * (D * 4 + 4) +
                T * 4 * -(-max(n for _, n in pairs) // 32), "flops": 4 * D * hq * seen}
    total = sum(p + n for p, n in pairs)
    old = 4 if case["decay"] else 0
    return {"bytes": keys * hkv * D + pages * (hkv * 4 + 4) + T * hq * (D * 2 + 4) +
            total * hkv * (4 + old), "flops": 2 * D * hq * seen}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _i32(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _table(perm, counts, first, cols):
    """Rows of a page table: sequence b's pages are perm[first[b]] and the counts[b] - 1 behind it."""
    at = torch.tensor(first, device="cuda")[:, None] + torch.arange(cols, device="cuda")
    used = torch.arange(cols, device="cuda") < torch.tensor(counts, device="cuda")[:, None]
    return torch.where(used, perm[at.clamp(max=perm.numel() - 1)], 0).to(torch.int32).contiguous()


def _batch(case, g, pairs, more=0):
    """Ragged batch over shuffled pages; `more` pages of the pool stay free."""
    order = torch.randperm(len(pairs), generator=g, device="cuda").tolist()
    pairs = [pairs[i] for i in order]
    page = case["page"]
    lens = [p + n for p, n in pairs]
    counts = [(v + page - 1) // page for v in lens]
    first = [sum(counts[:b]) for b in range(len(counts))]
    num_pages = sum(counts) + more + 3
    perm = torch.randperm(num_pages, generator=g, device="cuda").to(torch.int32)
    offsets = [0]
    for _, n in pairs:
        offsets.append(offsets[-1] + n)
    return {"q_offsets": _i32(offsets), "seq_lens": _i32(lens), "order": order,
            "page_table": _table(perm, counts, first, max(counts)), "num_pages": num_pages,
            "free": perm[sum(counts):], "T": offsets[-1], "new": [n for _, n in pairs],
            "lens": lens, "max_n": max(n for _, n in pairs), "max_len": max(lens)}


def _cache(case, g, num_pages):
    """E4M3 codes with the spread of unit-variance keys and values, and power-of-two scales of
    each page and head (some heads twice or four times louder than others)."""
    shape = (num_pages, case["kv_heads"], case["page"], case["D"])
    out = []
    for _ in range(2):
        codes = torch.empty(shape, dtype=torch.uint8, device="cuda")
        for part in codes.split(max(1, (1 << 27) // codes[0].numel())):
            part.copy_((torch.randn(part.shape, generator=g, device="cuda") * 90)
                       .clamp_(-448, 448).to(_F8).view(torch.uint8))
        scales = torch.exp2(torch.randint(-8, -5, shape[:2], generator=g, device="cuda").float())
        out += [codes, scales]
    return {"k_codes": out[0], "k_scales": out[1], "v_codes": out[2], "v_scales": out[3]}


def _stale(s, case):
    """Slots past a sequence's end hold whatever was there: here NaN codes."""
    page = case["page"]
    b = torch.arange(case["B"], device="cuda")
    last = s["page_table"][b, ((s["seq_lens"] - 1) // page).long()].long()
    past_end = torch.arange(page, device="cuda") >= ((s["seq_lens"] - 1) % page + 1)[:, None]
    for plane in ("k_codes", "v_codes"):
        pages = s[plane][last]
        pages.masked_fill_(past_end[:, None, :, None], 0x7F)
        s[plane][last] = pages


def _trees(new, seed):
    """Trees of drafted tokens as rows of ancestor bits: node 0 is the last token of the text, and
    a node hangs below one of the nodes before it, more often below a recent one. Level by level,
    as drafts are made."""
    rng = random.Random(seed)
    words = -(-max(new) // 32)
    rows = []
    for n in new:
        level, parents = [0], [-1]
        for _ in range(1, n):
            a = max(rng.randrange(len(level)), rng.randrange(len(level)))
            parents.append(a)
            level.append(level[a] + 1)
        order = sorted(range(n), key=lambda i: level[i])        # stable: by level, then as drafted
        place = {node: i for i, node in enumerate(order)}
        bits = [0] * n
        for i, node in enumerate(order):
            bits[i] = 1 << i | (bits[place[parents[node]]] if node else 0)
        rows += [[(v >> 32 * w) & 0xFFFFFFFF for w in range(words)] for v in bits]
    t = torch.tensor(rows, dtype=torch.int64)
    return torch.where(t >= 1 << 31, t - (1 << 32), t).to(torch.int32).cuda()


def _kept_of(n):
    """Tokens of a tree of n nodes that a step accepts, the root among them."""
    return min(n, 1 + int(math.log2(n) * 0.8))


def _paths(new, seed):
    """Accepted paths: the root, then nodes of later levels (which come behind as many nodes as the
    path has), ascending."""
    rng = random.Random(seed)
    width = max(_kept_of(n) for n in new)
    rows = []
    for n in new:
        k = _kept_of(n)
        later = range(k, n)
        path = [0] + sorted(rng.sample(later, min(k - 1, len(later))))
        rows.append(path + [-1] * (width - len(path)))
    return _i32(rows), _i32([sum(v >= 0 for v in r) for r in rows])


def _sees(s, case, b, rows=None):
    """Which of sequence b's tokens its new tokens see, [n, length], by the definitions."""
    length, n, w = s["lens"][b], s["new"][b], case["window"]
    start = length - n
    j = torch.arange(length, device="cuda")
    if rows is None:                       # causal
        place = torch.arange(start, length, device="cuda")[:, None]
        sees = j <= place
        return sees & (j > place - w) if w else sees
    bit = torch.arange(n, device="cuda")
    mine = (rows.long()[:, bit // 32] >> (bit % 32)) & 1 != 0
    sees = torch.cat((torch.ones(n, start, dtype=torch.bool, device="cuda"), mine), 1)
    if w:                                  # the last w tokens of the row's own chain
        from_end = sees.flip(1).cumsum(1).flip(1)
        sees &= from_end <= w
    return sees


def prepare(case, seed):
    g = _gen(seed)
    s = {"case": case}
    op = case["op"]
    if op == "norm":
        _prepare_norm(s, case, g)
    elif op == "evict":
        _prepare_evict(s, case, g)
    else:
        s.update(_batch(case, g, _lengths(case)))
        s.update(_cache(case, g, s["num_pages"]))
    if op == "keep":
        s["keep"], s["n_keep"] = _paths(s["new"], seed)
        s["new_lens"] = torch.empty_like(s["seq_lens"])
    if op in ("tree", "weights"):
        _stale(s, case)
        s["q"] = torch.randn(s["T"], case["q_heads"], case["D"], generator=g, device="cuda") \
            .to(_DT[case["dtype"]])
        s["scale"] = case["D"] ** -0.5
    if op == "tree":
        s["mask"] = _trees(s["new"], seed)
        s["out"] = torch.empty_like(s["q"])
        s["lse"] = torch.empty(s["T"], case["q_heads"], device="cuda")
    if op == "weights":
        # the attention call before this one left each row's log-sum
        s["lse"] = torch.empty(s["T"], case["q_heads"], device="cuda")
        at = 0
        for b, n in enumerate(s["new"]):
            for h in range(case["kv_heads"]):
                rows, score = _scores(s, case, b, at, h, torch.float32)
                score = score.masked_fill_(~_sees(s, case, b)[:, None], float("-inf"))
                s["lse"][at:at + n, rows] = torch.logsumexp(score, 2)
            at += n
        shape = (s["num_pages"], case["kv_heads"], case["page"])
        s["weights"] = torch.rand(shape, generator=g, device="cuda").square_()
        s["after"] = torch.zeros(shape, device="cuda")
    if own:
        _prepare_own(s)
    return s


def _scores(s, case, b, at, h, dtype):
    """Rows of key head h of sequence b (token rows from `at`) against its keys, [n, group, length]."""
    group, length = case["q_heads"] // case["kv_heads"], s["lens"][b]
    pages = s["page_table"][b, :-(-length // case["page"])].long()
    k = s["k_codes"][pages, h].view(_F8).to(dtype) * s["k_scales"][pages, h].to(dtype)[:, None, None]
    k = k.flatten(0, 1)[:length]
    rows = slice(h * group, (h + 1) * group)
    q = s["q"][at:at + s["new"][b], rows].to(dtype)
    return rows, torch.matmul(q, k.t()) * s["scale"]


def _prepare_evict(s, case, g):
    pairs = _evict_lengths(case)
    page = case["page"]
    pages_of = [-(-min(n, k) // page) for n, k in pairs]
    s.update(_batch(case, g, [(n, 0) for n, _ in pairs], more=sum(pages_of)))
    s.update(_cache(case, g, s["num_pages"]))
    budgets = [pairs[i][1] for i in s["order"]]
    counts = [pages_of[i] for i in s["order"]]
    s["budget"] = _i32(budgets)
    s["most"] = case["budget"]
    s["dst_table"] = _table(s["free"], counts, [sum(counts[:b]) for b in range(len(counts))], max(counts))
    # a few tokens hold most of the attention, and many have had none that a float shows
    shape = (s["num_pages"], case["kv_heads"], page)
    w = torch.exp(3 * torch.randn(shape, generator=g, device="cuda"))
    none = torch.rand(shape, generator=g, device="cuda") < 0.2
    s["weights"] = torch.where(none, torch.zeros_like(w), w)
    s["kept"] = torch.empty(case["B"], case["kv_heads"], s["most"], dtype=torch.int32, device="cuda")
    s["new_lens"] = torch.empty_like(s["seq_lens"])


def _prepare_norm(s, case, g):
    T, H = case["T"], case["H"]
    s["y"] = (torch.randn(T, H, generator=g, device="cuda") * 2).to(_DT[case["y"]])
    s["residual"] = (torch.randn(T, H, generator=g, device="cuda") * 3).to(_DT[case["residual"]])
    s["out"] = torch.empty_like(s["residual"])
    s["normed"] = torch.empty(T, H, device="cuda", dtype=_DT[case["normed"]]) if case["pre"] else None
    for name in ("post", "pre"):
        w = (1 + 0.2 * torch.randn(H, generator=g, device="cuda")).to(torch.bfloat16)
        s[name] = w if case[name] else None
    shape = {"none": None, "token": (T, 1), "channel": (1, H), "full": (T, H)}[case["gate"]]
    s["gate"] = torch.randn(shape, generator=g, device="cuda") if shape else None


def _prepare_own(s):
    """The handles and workspaces that a serving loop keeps."""
    import nvfp4_grouped_gemm_gb300 as moe
    case, op = s["case"], s["case"]["op"]
    s["moe"] = moe
    if op == "norm":
        return
    s["cache"] = moe.PagedKvCache(s["k_codes"], s["v_codes"], s["k_scales"], s["v_scales"])
    s["batch"] = moe.SeqBatch(s["q_offsets"], s["seq_lens"], s["page_table"])
    if op == "tree":
        n = moe.attention_workspace_bytes(case["q_heads"], case["kv_heads"], case["D"])
    elif op == "weights":
        n = moe.kv_weights_workspace_bytes(s["T"], case["q_heads"], case["kv_heads"], case["D"])
    elif op == "evict":
        n = moe.kv_evict_workspace_bytes(case["B"], case["kv_heads"])
    else:
        n = moe.kv_keep_workspace_bytes()
    s["ws"] = torch.zeros(n, dtype=torch.uint8, device="cuda")


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------
def run(state):
    op = state["case"]["op"]
    if own:
        return _OWN[op](state)
    return _PLAIN[op](state)


def _tree_own(s):
    s["moe"].moe_attention_tree_e4m3(s["q"], s["cache"], s["batch"], s["mask"], s["out"], s["ws"],
                                     scale=s["scale"], window=s["case"]["window"], lse=s["lse"])
    return {"out": s["out"], "lse": s["lse"]}


def _weights_own(s):
    s["moe"].moe_kv_weights_e4m3(s["q"], s["lse"], s["cache"], s["batch"], s["weights"], s["ws"],
                                 out=s["after"], scale=s["scale"], window=s["case"]["window"],
                                 decay=s["case"]["decay"])
    return s["after"]


def _evict_own(s):
    case = s["case"]
    s["moe"].moe_kv_evict_e4m3(s["cache"], s["batch"], s["weights"], s["dst_table"], s["kept"],
                               s["new_lens"], s["ws"], budgets=s["budget"], first=case["first"],
                               recent=case["recent"])
    return _evict_outputs(s)


def _planes(s):
    return {"k": s["k_codes"].view(_F8), "k_scales": s["k_scales"], "v": s["v_codes"].view(_F8),
            "v_scales": s["v_scales"], "new_lens": s["new_lens"]}


def _evict_outputs(s):
    return {**_planes(s), "weights": s["weights"], "kept": s["kept"]}


def _keep_own(s):
    s["moe"].moe_kv_keep_e4m3(s["cache"], s["batch"], s["keep"], s["n_keep"], s["new_lens"], s["ws"])
    return _planes(s)


def _norm_own(s):
    case = s["case"]
    s["moe"].moe_residual_norm(s["y"], s["residual"], s["out"], normed=s["normed"],
                               post_weight=s["post"], pre_weight=s["pre"], gate=s["gate"],
                               gate_sigmoid=case["sigmoid"], scale=case["scale"], eps=1e-6)
    return _norm_outputs(s)


def _norm_outputs(s):
    return {"out": s["out"]} if s["normed"] is None else {"out": s["out"], "normed": s["normed"]}


_OWN = {"tree": _tree_own, "weights": _weights_own, "evict": _evict_own, "keep": _keep_own,
        "norm": _norm_own}


# ---- plain forms ----------------------------------------------------------
def _rows_of(s):
    """For each new token: its sequence and its number among the sequence's new tokens."""
    t = torch.arange(s["T"], device="cuda")
    off = s["q_offsets"].long()
    b = torch.searchsorted(off[1:].contiguous(), t, right=True)
    return b, t - off[b]


def _gathered(s, codes, scales):
    """A plane as [B, heads, padded length, D] in 32 bits, through the page table."""
    table = s["page_table"].long()
    x = codes[table].view(_F8).float() * scales[table][..., None, None]
    return x.transpose(1, 2).flatten(2, 3)


def _padded_scores(s):
    """Scores [B, key heads, group, n, padded length] of the new tokens against all keys."""
    case = s["case"]
    hq, hkv, D = case["q_heads"], case["kv_heads"], case["D"]
    b, i = _rows_of(s)
    B, n = case["B"], s["max_n"]
    q = torch.zeros(B, n, hq, D, device="cuda")
    q[b, i] = s["q"].float()
    q = q.view(B, n, hkv, hq // hkv, D).permute(0, 2, 3, 1, 4).flatten(2, 3)
    k = _gathered(s, s["k_codes"], s["k_scales"])
    scores = torch.matmul(q, k.transpose(-1, -2)).view(B, hkv, hq // hkv, n, k.shape[2])
    return b, i, scores * s["scale"]


def _tree_plain(s):
    case = s["case"]
    hkv, D, B, n, w = case["kv_heads"], case["D"], case["B"], s["max_n"], case["window"]
    b, i, scores = _padded_scores(s)
    L = scores.shape[-1]
    lens = s["seq_lens"].long()
    start = lens - (s["q_offsets"][1:] - s["q_offsets"][:-1]).long()
    # the tree's bits at the places of the new tokens
    j = torch.arange(L, device="cuda")
    c = j - start[:, None]                                             # [B, L]
    rows = torch.zeros(B, n, s["mask"].shape[1], dtype=torch.long, device="cuda")
    rows[b, i] = s["mask"].long()
    inside = c.clamp(0, 32 * rows.shape[2] - 1)
    bits = torch.gather(rows, 2, (inside // 32)[:, None].expand(-1, n, -1)) >> (inside % 32)[:, None]
    sees = torch.where((c < 0)[:, None], torch.ones_like(bits), bits & 1) != 0
    sees &= (j < lens[:, None])[:, None]
    if w:
        sees &= sees.flip(2).cumsum(2).flip(2) <= w
    scores = torch.where(sees[:, None, None], scores, float("-inf"))
    top = scores.amax(-1, keepdim=True)
    p = torch.exp(scores - torch.where(top > float("-inf"), top, torch.zeros_like(top)))
    del scores
    total = p.sum(-1, keepdim=True)
    v = _gathered(s, s["v_codes"], s["v_scales"])
    v = torch.where((j < lens[:, None])[:, None, :, None], v, 0)
    o = torch.matmul(p.flatten(2, 3), v).view(B, hkv, -1, n, D)
    o = torch.where(total > 0, o / total, torch.zeros_like(o))
    lse = (top + total.log()).squeeze(-1).permute(0, 3, 1, 2).flatten(2)
    s["out"].copy_(o.permute(0, 3, 1, 2, 4).flatten(2, 3)[b, i])
    s["lse"].copy_(lse[b, i])
    return {"out": s["out"], "lse": s["lse"]}


def _weights_plain(s):
    case = s["case"]
    B, n, w, page = case["B"], s["max_n"], case["window"], case["page"]
    hkv, hq = case["kv_heads"], case["q_heads"]
    b, i, scores = _padded_scores(s)
    lens = s["seq_lens"].long()
    start = lens - (s["q_offsets"][1:] - s["q_offsets"][:-1]).long()
    j = torch.arange(scores.shape[-1], device="cuda")
    at = torch.full((B, n), -1, device="cuda", dtype=torch.long)
    at[b, i] = start[b] + i
    sees = j <= at[..., None]
    if w:
        sees &= j > at[..., None] - w
    lse = torch.zeros(B, n, hq, device="cuda")
    lse[b, i] = s["lse"]
    lse = lse.view(B, n, hkv, -1).permute(0, 2, 3, 1)[..., None]
    p = torch.where(sees[:, None, None], torch.exp(scores - lse), torch.zeros_like(scores))
    add = p.sum((2, 3))                                                # [B, key heads, length]
    pages = s["page_table"].long()[:, j // page]                       # [B, length]
    old = s["weights"][pages, :, (j % page).expand_as(pages)].transpose(1, 2) * case["decay"]
    old = torch.where((j < start[:, None])[:, None], old, torch.zeros_like(old))
    there = j < lens[:, None]
    bb, jj = there.nonzero(as_tuple=True)
    s["after"][pages[bb, jj], :, jj % page] = (old + add)[bb, :, jj]
    return s["after"]


def _moved(codes, old, new):
    """Codes under another scale: values in 32 bits, rounded once to E4M3."""
    return (codes.view(_F8).float() * (old / new)[..., None]).to(_F8).view(torch.uint8)


def _evict_plain(s):
    case = s["case"]
    B, hkv, page, K = case["B"], case["kv_heads"], case["page"], s["most"]
    lens = s["seq_lens"].long()
    keep = torch.minimum(lens, s["budget"].long())
    j = torch.arange(s["page_table"].shape[1] * page, device="cuda")
    w = s["weights"][s["page_table"].long()].transpose(1, 2).flatten(2)            # [B, heads, length]
    recent = torch.minimum(keep, torch.full_like(keep, case["recent"]))
    first = torch.minimum(keep - recent, torch.full_like(keep, case["first"]))
    safe = (j < first[:, None]) | (j >= (lens - recent)[:, None])
    w = torch.where(safe[:, None], float("inf"), w)
    w = torch.where((j < lens[:, None])[:, None], w, float("-inf"))
    order = torch.sort(w, dim=2, descending=True, stable=True).indices
    if order.shape[2] < K:
        order = torch.cat((order, order.new_zeros(B, hkv, K - order.shape[2])), 2)
    slot = torch.arange(K, device="cuda")
    there = (slot < keep[:, None])[:, None].expand(B, hkv, K)
    kept = torch.where(there, order[..., :K], 1 << 40).sort(2).values
    kept = torch.where(there, kept, -1)
    s["kept"].copy_(kept)
    s["new_lens"].copy_(keep)
    b, h, i = there.nonzero(as_tuple=True)
    src = kept[b, h, i]
    from_page = s["page_table"][b, src // page].long()
    to_page = s["dst_table"][b, i // page].long()
    for name in ("k", "v"):
        codes, scales = s[name + "_codes"], s[name + "_scales"]
        old = scales[from_page, h]
        new = torch.zeros_like(scales)
        new.view(-1).scatter_reduce_(0, to_page * hkv + h, old, "amax")
        new = new[to_page, h]
        codes[to_page, h, i % page] = _moved(codes[from_page, h, src % page], old, new)
        scales[to_page, h] = new
    s["weights"][to_page, h, i % page] = s["weights"][from_page, h, src % page]
    return _evict_outputs(s)


def _keep_plain(s):
    page, hkv = s["case"]["page"], s["case"]["kv_heads"]
    lens = s["seq_lens"].long()
    start = lens - (s["q_offsets"][1:] - s["q_offsets"][:-1]).long()
    n_keep = s["n_keep"].long()
    b, i = (torch.arange(s["keep"].shape[1], device="cuda") < n_keep[:, None]).nonzero(as_tuple=True)
    src, dst = start[b] + s["keep"].long()[b, i], start[b] + i
    from_page = s["page_table"][b, src // page].long()
    to_page = s["page_table"][b, dst // page].long()
    h = torch.arange(hkv, device="cuda")
    for name in ("k", "v"):
        codes, scales = s[name + "_codes"], s[name + "_scales"]
        old = scales.clone()
        scales.view(-1).scatter_reduce_(0, (to_page[:, None] * hkv + h).flatten(),
                                        old[from_page].flatten(), "amax")
        data = codes[from_page, :, src % page]
        touched = to_page.unique()
        codes[touched] = _moved(codes[touched], old[touched][..., None], scales[touched][..., None])
        codes[to_page, :, dst % page] = _moved(data, old[from_page], scales[to_page])
    s["new_lens"].copy_(start + n_keep)
    return _planes(s)


def _rms(x, w):
    return x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6) * w.float()


def _norm_plain(s):
    z = s["y"].float()
    if s["post"] is not None:
        z = _rms(z, s["post"])
    if s["gate"] is not None:
        z = z * (1 / (1 + torch.exp(-s["gate"])) if s["case"]["sigmoid"] else s["gate"])
    r = s["residual"].float() + s["case"]["scale"] * z
    s["out"].copy_(r)
    if s["normed"] is not None:
        s["normed"].copy_(_rms(r, s["pre"]))
    return _norm_outputs(s)


_PLAIN = {"tree": _tree_plain, "weights": _weights_plain, "evict": _evict_plain,
          "keep": _keep_plain, "norm": _norm_plain}


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------
def exact(case, seed):
    global own
    was, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = was
    return {"tree": _tree_exact, "weights": _weights_exact, "evict": _evict_exact,
            "keep": _keep_exact, "norm": _norm_exact}[case["op"]](case, s)


def _e4m3_table():
    bytes_ = torch.arange(256, dtype=torch.uint8, device="cuda")
    return bytes_.view(_F8).double()


def _near(x):
    """Nearest E4M3 value, ties to the even code."""
    a = x.abs().clamp(2.0 ** -60)
    step = torch.exp2(torch.floor(torch.log2(a)).clamp(min=-6) - 3)
    return torch.round(x / step) * step


def _tree_exact(case, s):
    grid = _e4m3_table()
    hq, D = case["q_heads"], case["D"]
    out = torch.zeros(s["T"], hq, D, dtype=torch.float64, device="cuda")
    lse = torch.zeros(s["T"], hq, dtype=torch.float64, device="cuda")
    at = 0
    for b, n in enumerate(s["new"]):
        length = s["lens"][b]
        hidden = ~_sees(s, case, b, s["mask"][at:at + n])
        pages = s["page_table"][b, :-(-length // case["page"])].long()
        for h in range(case["kv_heads"]):
            v = (grid[s["v_codes"][pages, h].long()] * s["v_scales"][pages, h].double()[:, None, None])
            v = v.flatten(0, 1)[:length]
            rows, score = _scores(s, case, b, at, h, torch.float64)
            score = score.masked_fill(hidden[:, None], float("-inf"))
            lse[at:at + n, rows] = torch.logsumexp(score, 2)
            out[at:at + n, rows] = torch.softmax(score, 2) @ v
        at += n
    return {"out": out, "lse": lse}


def _weights_exact(case, s):
    page = case["page"]
    after = torch.zeros(s["weights"].shape, dtype=torch.float64, device="cuda")
    at = 0
    for b, n in enumerate(s["new"]):
        length = s["lens"][b]
        j = torch.arange(length, device="cuda")
        pages = s["page_table"][b, j // page].long()
        sees = _sees(s, case, b)
        for h in range(case["kv_heads"]):
            rows, score = _scores(s, case, b, at, h, torch.float64)
            p = torch.exp(score - s["lse"][at:at + n, rows].double()[..., None])
            add = (p * sees[:, None]).sum((0, 1))
            old = s["weights"][pages, h, j % page].double() * case["decay"]
            old[length - n:] = 0
            after[pages, h, j % page] = old + add
        at += n
    return after


def _evict_exact(case, s):
    grid, page = _e4m3_table(), case["page"]
    planes = {n: (grid[s[n + "_codes"].long()], s[n + "_scales"].double()) for n in ("k", "v")}
    weights = s["weights"].double()
    kept = torch.full(s["kept"].shape, -1, dtype=torch.int64, device="cuda")
    budgets = s["budget"].tolist()
    for b, length in enumerate(s["lens"]):
        keep = min(length, budgets[b])
        recent = min(case["recent"], keep)
        first = min(case["first"], keep - recent)
        j = torch.arange(length, device="cuda")
        pages = s["page_table"][b, j // page].long()
        for h in range(case["kv_heads"]):
            rest = s["weights"][pages, h, j % page][first:length - recent].double()
            best = torch.sort(rest, descending=True, stable=True).indices[:keep - recent - first]
            chosen = torch.cat((j[:first], first + best.sort().values, j[length - recent:]))
            kept[b, h, :keep] = chosen
            for p in range(-(-keep // page)):
                src = chosen[p * page:(p + 1) * page]
                to, from_page, k = int(s["dst_table"][b, p]), pages[src], src.numel()
                weights[to, h, :k] = s["weights"][from_page, h, src % page].double()
                for name, (values, scales) in planes.items():
                    old = s[name + "_scales"][from_page, h].double()
                    codes = grid[s[name + "_codes"][from_page, h, src % page].long()]
                    scales[to, h] = old.max()
                    values[to, h, :k] = _near(codes * (old / old.max())[:, None])
    lens = torch.tensor([min(n, k) for n, k in zip(s["lens"], budgets)], device="cuda")
    return {"k": planes["k"][0], "k_scales": planes["k"][1], "v": planes["v"][0],
            "v_scales": planes["v"][1], "new_lens": lens, "weights": weights, "kept": kept}


def _keep_exact(case, s):
    grid, page = _e4m3_table(), case["page"]
    planes = {n: (grid[s[n + "_codes"].long()], s[n + "_scales"].double()) for n in ("k", "v")}
    table, counts, keep = s["page_table"].tolist(), s["n_keep"].tolist(), s["keep"].tolist()
    lens = []
    for b, length in enumerate(s["lens"]):
        start = length - s["new"][b]
        lens.append(start + counts[b])
        moves = [(start + keep[b][i], start + i) for i in range(counts[b])]
        for name, (values, scales) in planes.items():
            before = {p: (values[table[b][p]].clone(), scales[table[b][p]].clone())
                      for p in {v // page for m in moves for v in m}}
            for p in sorted({to // page for _, to in moves}):
                into = [(a, to) for a, to in moves if to // page == p]
                new = before[p][1]
                for a, _ in into:
                    new = torch.maximum(new, before[a // page][1])
                held = _near(before[p][0] * (before[p][1] / new)[:, None, None])
                for a, to in into:
                    was, scale = before[a // page]
                    held[:, to % page] = _near(was[:, a % page] * (scale / new)[:, None])
                values[table[b][p]], scales[table[b][p]] = held, new
    return {"k": planes["k"][0], "k_scales": planes["k"][1], "v": planes["v"][0],
            "v_scales": planes["v"][1], "new_lens": torch.tensor(lens, device="cuda")}


def _norm_exact(case, s):
    z = s["y"].double()
    if case["post"]:
        z = z / torch.sqrt((z * z).sum(1, keepdim=True) / case["H"] + 1e-6) * s["post"].double()
    if case["gate"] != "none":
        gate = s["gate"].double()
        z = z * (torch.sigmoid(gate) if case["sigmoid"] else gate)
    r = s["residual"].double() + z * case["scale"]
    if not case["pre"]:
        return {"out": r}
    n = r / torch.sqrt((r * r).sum(1, keepdim=True) / case["H"] + 1e-6) * s["pre"].double()
    return {"out": r, "normed": n}
