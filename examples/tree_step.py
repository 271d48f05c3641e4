"""One decoder block served with trees of drafted tokens and a bounded cache, on NVFP4 weights.

A step scores every sequence's tree together: norm (moe_residual_norm), q/k/v projection
(moe_linear_nvfp4), append of keys and values at the places behind the text, rotated by each node's
depth (moe_kv_append_rope_e4m3 with positions), attention in which a node sees the text and its
ancestors (moe_attention_tree_e4m3), output projection, residual and norm, the routed MoE layer
(MoeLayer), residual and norm, and the head.  A token is drawn for every node (moe_verify_draft without
drafts); the path that the draws follow is kept in the cache (moe_kv_keep_e4m3), its tokens' attention is
added to the cached tokens' weights (moe_kv_weights_e4m3), and a sequence that outgrows its budget is
cut to the tokens with the largest weights (moe_kv_evict_e4m3).  Weights are random; a tree's branches
are what followed the last token at its latest occurrences.

    python examples/tree_step.py
"""
from __future__ import annotations

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import nvfp4_grouped_gemm_gb300 as moe  # noqa: E402
from speculative_step import Block  # noqa: E402


class TreeBlock(Block):
    """The block of the speculative example with its norms and residuals in single passes."""

    def __init__(self, **kw):
        super().__init__(**kw)
        ones = torch.ones(self.hidden, device="cuda", dtype=torch.bfloat16)
        self.norms = [ones.clone() for _ in range(3)]

    def normed(self, y, residual, weight):
        """residual + y (residual itself, in place) and its norm in bf16."""
        out = torch.empty(residual.shape, dtype=torch.bfloat16, device="cuda")
        moe.moe_residual_norm(y, residual, None if y is None else residual, normed=out, pre_weight=weight)
        return out

    def tree_logits(self, tokens, cache, batch, positions, mask):
        """Logits of the batch's new tokens, and the queries and log sums of their attention."""
        x = self.embedding[tokens].contiguous()
        rows = self.qkv.forward(self.normed(None, x, self.norms[0]))
        d = self.head_dim
        q, k, v = (part.view(-1, part.shape[1] // d, d) for part in
                   rows.split([self.q_heads * d, self.kv_heads * d, self.kv_heads * d], 1))
        q = q.contiguous()
        moe.moe_kv_append_rope_e4m3(cache, batch, k, v, self.cos, self.sin, self.ws, q=q, positions=positions)
        seen = torch.empty_like(q)
        lse = torch.empty(q.shape[:2], device="cuda")
        moe.moe_attention_tree_e4m3(q, cache, batch, mask, seen, self.ws, lse=lse)
        h = self.normed(self.o.forward(seen.flatten(1)), x, self.norms[1])
        y = self.layer.forward(h, logits=h.float() @ self.router.t())
        return self.head.forward(self.normed(y, x, self.norms[2])), q, lse


class TreeServer:
    """Sequences over one paged cache; every step scores a tree each, keeps the path that the drawn
    tokens follow, and cuts sequences of more than `budget` tokens down to it."""

    def __init__(self, block, prompts, page=16, nodes=8, budget=64, recent=16):
        self.block, self.nodes, self.budget, self.recent, self.page = block, nodes, budget, recent, page
        B = self.B = len(prompts)
        self.per = -(-(max(budget, max(map(len, prompts))) + 2 * nodes) // page)
        self.cache = moe.PagedKvCache.allocate(2 * B * self.per, block.kv_heads, page, block.head_dim)
        self.weights = torch.zeros(2 * B * self.per, block.kv_heads, page, device="cuda")
        # a sequence has two sets of pages, one in use and one that an eviction copies into
        order = torch.randperm(2 * B * self.per, generator=block.g, device="cuda").to(torch.int32)
        self.tables = order.view(2, B, self.per)
        self.table, self.other = self.tables[0].clone(), self.tables[1].clone()
        self.text = [list(p) for p in prompts]
        self.lens = [0] * B                     # cached tokens
        self.ws = torch.zeros(max(moe.kv_keep_workspace_bytes(), moe.verify_workspace_bytes(B * nodes, block.vocab),
                                  moe.kv_evict_workspace_bytes(B, block.kv_heads)), dtype=torch.uint8, device="cuda")
        # the prompts but for their last tokens, which open the first step: trees of one branch
        chains = [list(range(len(t) - 1)) for t in self.text]
        self._score([t[:-1] for t in self.text], [[i - 1 for i in c] for c in chains], [0] * B)
        self._commit(chains)
        self._weigh(chains, decay=0.0)

    def _batch(self, counts, lens):
        offsets = torch.tensor([0] + list(counts), dtype=torch.int32).cumsum(0, dtype=torch.int32)
        return moe.SeqBatch(offsets.cuda(), torch.tensor(lens, dtype=torch.int32).cuda(), self.table)

    def _score(self, tokens, parents, first):
        """Logits of each sequence's new tokens; parents[b][i] is a token's parent among them (-1: the
        text), and a root's position in the text is first[b]."""
        self.counts = [len(t) for t in tokens]
        self.batch = self._batch(self.counts, [n + c for n, c in zip(self.lens, self.counts)])
        words = -(-max(max(self.counts), 1) // 32)
        rows, positions = [], []
        for b, up in enumerate(parents):
            bits, depth = [], []
            for i, a in enumerate(up):
                bits.append(1 << i | (bits[a] if a >= 0 else 0))
                depth.append(depth[a] + 1 if a >= 0 else 0)
            rows += [[(v >> 32 * w) & 0xFFFFFFFF for w in range(words)] for v in bits]
            positions += [first[b] + d for d in depth]
        mask = torch.tensor(rows, dtype=torch.int64)
        mask = torch.where(mask >= 1 << 31, mask - (1 << 32), mask).to(torch.int32).cuda()
        flat = torch.tensor([t for s in tokens for t in s], device="cuda")
        logits, self.q, self.lse = self.block.tree_logits(
            flat, self.cache, self.batch, torch.tensor(positions, dtype=torch.int32).cuda(), mask)
        return logits

    def _commit(self, paths):
        """Keep each sequence's path of the tokens just scored."""
        width = max(len(p) for p in paths)
        keep = torch.tensor([p + [-1] * (width - len(p)) for p in paths], dtype=torch.int32).cuda()
        n_keep = torch.tensor([len(p) for p in paths], dtype=torch.int32).cuda()
        lens = torch.empty(self.B, dtype=torch.int32, device="cuda")
        moe.moe_kv_keep_e4m3(self.cache, self.batch, keep, n_keep, lens, self.ws)
        self.lens = lens.tolist()

    def _weigh(self, paths, decay=1.0):
        """Add the attention of the kept tokens' rows: the sequences' last tokens, which their nodes saw
        just as a chain does."""
        offsets = [0]
        for c in self.counts:
            offsets.append(offsets[-1] + c)
        at = torch.tensor([offsets[b] + i for b, p in enumerate(paths) for i in p], device="cuda")
        batch = self._batch([len(p) for p in paths], self.lens)
        q, lse = self.q[at].contiguous(), self.lse[at].contiguous()
        n = moe.kv_weights_workspace_bytes(q.shape[0], q.shape[1], self.block.kv_heads, self.block.head_dim)
        ws = torch.zeros(n, dtype=torch.uint8, device="cuda")
        moe.moe_kv_weights_e4m3(q, lse, self.cache, batch, self.weights, ws, decay=decay)

    def _tree(self, text):
        """Node 0 is the text's last token; below it what followed that token at its latest places."""
        tokens, parents = [text[-1]], [-1]
        at = [i for i in range(len(text) - 2, -1, -1) if text[i] == text[-1]]
        for i in at:
            node = 0
            for t in text[i + 1:i + 4]:
                if len(tokens) == self.nodes:
                    return tokens, parents
                found = next((j for j in range(len(tokens)) if parents[j] == node and tokens[j] == t), None)
                if found is None:
                    tokens.append(t)
                    parents.append(node)
                    found = len(tokens) - 1
                node = found
        return tokens, parents

    def step(self, u):
        """u [B * nodes] draws the nodes' tokens.  Returns how many drafted tokens each sequence took."""
        trees = [self._tree(t) for t in self.text]
        logits = self._score([t for t, _ in trees], [p for _, p in trees], [len(t) - 1 for t in self.text])
        probs = torch.softmax(logits, -1)
        T = probs.shape[0]
        ids = torch.empty(T, 1, dtype=torch.int32, device="cuda")
        none = torch.empty(T, 0, dtype=torch.int32, device="cuda")
        moe.moe_verify_draft(none, probs[:, None], torch.empty(T, 0, device="cuda"), u[:T].contiguous(), ids,
                             torch.empty(T, dtype=torch.int32, device="cuda"), self.ws)
        drawn, at, paths = ids[:, 0].tolist(), 0, []
        for b, (tokens, parents) in enumerate(trees):
            path = [0]
            while True:                        # follow the draws as long as a branch has them
                token = drawn[at + path[-1]]
                child = next((j for j in range(len(tokens)) if parents[j] == path[-1] and tokens[j] == token), None)
                self.text[b].append(token)
                if child is None:
                    break
                path.append(child)
            paths.append(path)
            at += len(tokens)
        self._commit(paths)
        self._weigh(paths)
        self.kept = None
        if max(self.lens) > self.budget:
            self._evict()
        return [len(p) - 1 for p in paths]

    def _evict(self):
        budgets = [self.budget if n > self.budget else -1 for n in self.lens]
        kept = torch.empty(self.B, self.block.kv_heads, self.budget, dtype=torch.int32, device="cuda")
        lens = torch.empty(self.B, dtype=torch.int32, device="cuda")
        moe.moe_kv_evict_e4m3(self.cache, self._batch([0] * self.B, self.lens), self.weights, self.other, kept, lens,
                              self.ws, budgets=torch.tensor(budgets, dtype=torch.int32).cuda(), first=1,
                              recent=self.recent)
        self.lens, self.kept = lens.tolist(), kept
        for b, budget in enumerate(budgets):
            if budget >= 0:
                row = self.table[b].clone()
                self.table[b], self.other[b] = self.other[b].clone(), row


def main(steps=12):
    g = torch.Generator(device="cuda").manual_seed(1)
    prompts = [[(7 * b + i * i) % 11 for i in range(20 + 9 * b)] for b in range(5)]
    server = TreeServer(TreeBlock(vocab=11), prompts)       # few words, so that branches are taken
    for i in range(steps):
        counts = server.step(torch.rand(server.B * server.nodes, generator=g, device="cuda"))
        print(f"step {i}: accepted {counts}, cached {server.lens}")
    print("device errors:", moe.get_device_error(server.block.ws), moe.get_device_error(server.ws))
    return server


if __name__ == "__main__":
    main()
