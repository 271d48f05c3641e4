"""One decoder block served with speculative decoding on NVFP4 weights.

A step scores the drafted tokens of every sequence together: q/k/v projection (moe_linear_nvfp4),
append of keys and values to the paged 8-bit cache with the rotary rotation
(moe_kv_append_rope_e4m3), attention over that cache (moe_attention_paged_e4m3), output projection,
routed MoE layer (MoeLayer), language-model head, and the verification of the drafts
(moe_verify_draft).  Weights are random; drafts repeat what followed the last token before.

    python examples/speculative_step.py
"""
from __future__ import annotations

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import nvfp4_grouped_gemm_gb300 as moe  # noqa: E402


def random_bank(g, E, rows, in_f, spread):
    """Random NVFP4 weights with a second-level scale that gives them about `spread`."""
    codes = torch.randint(0, 256, (E, rows, in_f // 2), generator=g, device="cuda", dtype=torch.uint8)
    scales = torch.randint(0x30, 0x39, (E, rows, in_f // 16), generator=g, device="cuda", dtype=torch.uint8)
    alpha = torch.full((E,), spread / 2.5, device="cuda")
    return moe.NvFp4Bank(codes, scales, alpha)


def rms_norm(x):
    x = x.float()
    return (x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6)).to(torch.bfloat16)


class Block:
    """Embedding, one attention + MoE block, and the language-model head."""

    def __init__(self, hidden=512, q_heads=8, kv_heads=2, head_dim=64, ff=128, experts=16, top_k=2,
                 vocab=1003, max_len=4096, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.g, self.hidden, self.head_dim = g, hidden, head_dim
        self.q_heads, self.kv_heads, self.vocab = q_heads, kv_heads, vocab
        width = (q_heads + 2 * kv_heads) * head_dim
        self.embedding = torch.randn(vocab, hidden, generator=g, device="cuda")
        self.qkv = moe.NvFp4Linear(random_bank(g, 1, width, hidden, hidden ** -0.5))
        self.o = moe.NvFp4Linear(random_bank(g, 1, hidden, q_heads * head_dim, hidden ** -0.5),
                                 torch.float32)
        self.router = torch.randn(experts, hidden, generator=g, device="cuda") * hidden ** -0.5
        self.layer = moe.MoeLayer(random_bank(g, experts, 2 * ff, hidden, hidden ** -0.5),
                                  random_bank(g, experts, hidden, ff, ff ** -0.5), top_k)
        self.head = moe.NvFp4Linear(random_bank(g, 1, vocab, hidden, 4 * hidden ** -0.5), torch.float32)
        inv = 10000.0 ** (-torch.arange(0, head_dim, 2, device="cuda", dtype=torch.float64) / head_dim)
        angle = torch.arange(max_len, device="cuda", dtype=torch.float64)[:, None] * inv
        self.cos, self.sin = angle.cos().float(), angle.sin().float()
        ws = max(moe.kv_append_workspace_bytes(),
                 moe.attention_workspace_bytes(q_heads, kv_heads, head_dim))
        self.ws = torch.zeros(ws, dtype=torch.uint8, device="cuda")

    def logits(self, tokens, cache, batch):
        """Logits of the batch's new tokens (flat, int64), their keys and values in the cache."""
        x = self.embedding[tokens]
        rows = self.qkv.forward(rms_norm(x))
        d = self.head_dim
        q, k, v = (part.view(-1, part.shape[1] // d, d) for part in
                   rows.split([self.q_heads * d, self.kv_heads * d, self.kv_heads * d], 1))
        moe.moe_kv_append_rope_e4m3(cache, batch, k, v, self.cos, self.sin, self.ws, q=q)
        seen = torch.empty(q.shape, dtype=q.dtype, device="cuda")
        moe.moe_attention_paged_e4m3(q, cache, batch, seen, self.ws)
        x = x + self.o.forward(seen.flatten(1))
        h = rms_norm(x)
        x = x + self.layer.forward(h, logits=h.float() @ self.router.t())
        return self.head.forward(rms_norm(x))


class Server:
    """Sequences over one paged cache; every step drafts, scores, verifies and moves on."""

    def __init__(self, block, prompts, page=16, max_len=512, drafts=3):
        self.block, self.drafts = block, drafts
        B, per = len(prompts), -(-max_len // page)
        self.cache = moe.PagedKvCache.allocate(B * per, block.kv_heads, page, block.head_dim)
        order = torch.randperm(B * per, generator=block.g, device="cuda").to(torch.int32)
        self.table = order.view(B, per).contiguous()
        self.text = [list(p) for p in prompts]
        self.lens = [0] * B
        self.draft_ws = torch.zeros(moe.verify_workspace_bytes(B, block.vocab), dtype=torch.uint8,
                                    device="cuda")
        # the prompts but for their last tokens, which open the first step
        self._score([t[:-1] for t in self.text])

    def _score(self, new):
        counts = [len(n) for n in new]
        self.lens = [n + c for n, c in zip(self.lens, counts)]
        offsets = torch.tensor([0] + counts, dtype=torch.int32).cumsum(0, dtype=torch.int32)
        batch = moe.SeqBatch(offsets.cuda(), torch.tensor(self.lens, dtype=torch.int32).cuda(), self.table)
        flat = torch.tensor([t for n in new for t in n], device="cuda")
        return self.block.logits(flat, self.cache, batch)

    def _lookup(self, text):
        """What followed the text's last token the time before (else the token itself)."""
        at = next((i for i in range(len(text) - 2, -1, -1) if text[i] == text[-1]), None)
        found = text[at + 1:at + 1 + self.drafts] if at is not None else []
        return found + [text[-1]] * (self.drafts - len(found))

    def step(self, u_accept, u_sample):
        """Returns how many drafted tokens each sequence accepted; one more is drawn for each."""
        B, n = len(self.text), self.drafts
        drafts = [self._lookup(t) for t in self.text]
        before = list(self.lens)
        logits = self._score([[t[-1]] + d for t, d in zip(self.text, drafts)])
        probs = torch.softmax(logits.view(B, n + 1, -1), -1)
        out = torch.empty(B, n + 1, dtype=torch.int32, device="cuda")
        accepted = torch.empty(B, dtype=torch.int32, device="cuda")
        moe.moe_verify_draft(torch.tensor(drafts, dtype=torch.int32).cuda(), probs, u_accept, u_sample,
                             out, accepted, self.draft_ws)
        got, counts = out.tolist(), accepted.tolist()
        for b in range(B):
            self.text[b] += got[b][:counts[b] + 1]
            # refused tokens' slots are written again by the next step
            self.lens[b] = before[b] + 1 + counts[b]
        return counts


def main(steps=8):
    g = torch.Generator(device="cuda").manual_seed(1)
    prompts = [[(7 * b + i * i) % 13 for i in range(5 + 9 * b)] for b in range(6)]
    server = Server(Block(vocab=13), prompts)      # few words, so that some drafts are accepted
    for i in range(steps):
        counts = server.step(torch.rand(6, server.drafts, generator=g, device="cuda"),
                             torch.rand(6, generator=g, device="cuda"))
        print(f"step {i}: accepted {counts}, lengths {server.lens}")
    errors = moe.get_device_error(server.block.ws), moe.get_device_error(server.draft_ws)
    print("device errors:", errors)
    return server


if __name__ == "__main__":
    main()
