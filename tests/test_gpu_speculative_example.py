"""The speculative-decoding example: its operators together, one block's logits against a float64
block over the same weights and the same 8-bit cache, and verification that follows the text."""
import importlib.util
import os

import numpy as np
import pytest
import torch

import nvfp4_grouped_gemm_gb300 as moe
from oracle import serving as oracle
from oracle.nvfp4 import dequant

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    spec = importlib.util.spec_from_file_location("speculative_step",
                                                  os.path.join(ROOT, "examples", "speculative_step.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def weights(bank, e=0):
    return torch.from_numpy(dequant(bank.codes[e].cpu().numpy(), bank.scales[e].cpu().numpy())) \
        * float(bank.alpha[e])


def norm(x):
    return x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6)


def reference_logits(block, tokens, cache, offsets, lens, table):
    """The block in float64, except that rows are rounded to bf16 where it stores bf16; the cache
    planes are read after the call, so they hold the call's own keys and values."""
    bf = lambda x: x.to(torch.bfloat16).double()      # noqa: E731
    x = block.embedding[tokens].double().cpu()
    rows = bf(bf(norm(x)) @ weights(block.qkv.bank).T)
    d, T = block.head_dim, len(tokens)
    q = rows[:, :block.q_heads * d].view(T, -1, d)
    place = np.concatenate([np.arange(lens[b] - (offsets[b + 1] - offsets[b]), lens[b])
                            for b in range(len(lens))])
    q = oracle.rotate(q.float().numpy(), block.cos.cpu().numpy()[place][:, None],
                      block.sin.cpu().numpy()[place][:, None], False)
    q = bf(torch.from_numpy(q))
    out = oracle.attention(q.numpy(), cache.k_codes.cpu().numpy(), cache.k_scales.cpu().numpy(),
                           cache.v_codes.cpu().numpy(), cache.v_scales.cpu().numpy(), offsets, lens,
                           table, d ** -0.5)[0]
    x = x + bf(torch.from_numpy(out)).flatten(1) @ weights(block.o.bank).T
    h = bf(norm(x))
    lo = h @ block.router.double().cpu().T
    top, ids = lo.topk(block.layer.k, 1)
    w = torch.softmax(top, 1)
    F = block.layer.F
    for t in range(T):
        for j in range(block.layer.k):
            gu = weights(block.layer.gate_up, int(ids[t, j])) @ h[t]
            x[t] += w[t, j] * (weights(block.layer.down, int(ids[t, j])) @
                               (torch.nn.functional.silu(gu[:F]) * gu[F:]))
    return bf(norm(x)) @ weights(block.head.bank).T


def test_a_block_s_logits_against_float64(example):
    block = example.Block(seed=3)
    page, lens = 16, [9, 40, 1]
    cache = moe.PagedKvCache.allocate(16, block.kv_heads, page, block.head_dim)
    table = np.random.default_rng(0).permutation(12).reshape(3, 4).astype(np.int32)
    tokens = torch.arange(sum(lens), device="cuda") * 13 % block.vocab
    offsets = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
    batch = moe.SeqBatch(torch.from_numpy(offsets).cuda(), torch.tensor(lens, dtype=torch.int32).cuda(),
                         torch.from_numpy(table).cuda())
    got = block.logits(tokens, cache, batch).double().cpu()
    want = reference_logits(block, tokens, cache, offsets, lens, table)
    assert moe.get_device_error(block.ws) == 0
    # a bf16 rounding that falls the other way moves a row by 2^-8 of one value in hundreds; a
    # router near-tie would show as an error of the order of the logits themselves
    rel = (got - want).norm(dim=1) / want.norm(dim=1)
    assert float(rel.max()) < 0.02, rel


def test_steps_move_along_the_text(example):
    server = example.main(steps=4)
    for text, n in zip(server.text, server.lens):
        assert n == len(text) - 1                     # the last token opens the next step
        assert all(0 <= t < server.block.vocab for t in text)


def test_random_numbers_of_zero_accept_every_likely_draft(example):
    """With u = 0 a draft is refused only at probability 0, so every step keeps all of them."""
    server = example.Server(example.Block(seed=5), [[1, 2, 3], [4, 5, 6, 7]], drafts=2)
    counts = server.step(torch.zeros(2, 2, device="cuda"), torch.full((2,), 0.5, device="cuda"))
    assert counts == [2, 2]
