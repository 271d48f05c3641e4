"""The example of trees and a bounded cache: the operators together. Every cached key is the key of the text's
token that should be there, rotated by its place in the text, whatever paths were kept and whatever was
evicted; and rows' weights sum to one each."""
import importlib.util
import os

import numpy as np
import pytest
import torch

import nvfp4_grouped_gemm_gb300 as moe
from oracle import serving as oracle
from oracle.nvfp4 import dequant
from serving_util import Batch, activations, cache_planes, device_cache, zeros_ws

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    spec = importlib.util.spec_from_file_location("tree_step", os.path.join(ROOT, "examples", "tree_step.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def key_rows(block):
    """Every token's keys [vocab, kv_heads, dim] before rotation, in float64, and a bound of their error: the
    normed row and the projection's result are bf16 (each off by at most 2^-8 of the value)."""
    x = block.embedding.double().cpu()
    x = x * torch.rsqrt(x.square().mean(1, keepdim=True) + 1e-6)
    bank = block.qkv.bank
    w = torch.from_numpy(dequant(bank.codes[0].cpu().numpy(), bank.scales[0].cpu().numpy())) * float(bank.alpha[0])
    d, hq, hk = block.head_dim, block.q_heads, block.kv_heads
    w = w[hq * d:(hq + hk) * d].double()
    y, mag = x @ w.T, x.abs() @ w.abs().T
    err = 2.0 ** -8 * 1.01 * (mag + y.abs()) + 2.0 ** -16 * mag
    return y.numpy().reshape(-1, hk, d), err.numpy().reshape(-1, hk, d)


def check_keys(server, origin, keys, errs):
    """Cached keys against the text: a rotated pair is off by both values' errors, and a code by half a step
    of E4M3 (2^-4 of the value, 2^-10 of the scale below its least normal) each time it was rounded: at the
    append, and when its page's scale grew or it moved to a page with a larger one."""
    block, page = server.block, server.page
    codes, scales = server.cache.k_codes.cpu().numpy(), server.cache.k_scales.cpu().numpy()
    table = server.table.cpu().numpy()
    cos, sin = block.cos.cpu().numpy(), block.sin.cpu().numpy()
    half = block.head_dim // 2
    for b in range(server.B):
        for h in range(block.kv_heads):
            at = np.array(origin[b][h])
            assert len(at) == server.lens[b]
            tok = np.array(server.text[b])[at]
            k, e = keys[tok, h], errs[tok, h]
            want = oracle.rotate(k.astype(np.float32), cos[at], sin[at], False).astype(np.float64)
            err = np.concatenate([e[:, :half] + e[:, half:]] * 2, 1) + 2.0 ** -20 * np.abs(k).max()
            j = np.arange(len(at))
            pages = table[b, j // page]
            scale = scales[pages, h][:, None].astype(np.float64)
            got = oracle.E4M3[codes[pages, h, j % page]] * scale
            tol = err
            for _ in range(4):
                tol = tol + 2.0 ** -4 * (np.abs(want) + tol) + 2.0 ** -10 * scale
            assert np.all(np.abs(got - want) <= tol), (b, h)


@pytest.mark.parametrize("page,budget", [(16, 10000), (16, 48), (32, 40), (64, 33)])
def test_the_cache_holds_what_the_text_says(example, page, budget):
    prompts = [[(5 * b + i * i) % 9 for i in range(11 + 13 * b)] for b in range(5)]
    server = example.TreeServer(example.TreeBlock(vocab=9, seed=3), prompts, page=page, nodes=9,
                                budget=min(budget, 200), recent=8)
    keys, errs = key_rows(server.block)
    origin = [[list(range(n)) for _ in range(server.block.kv_heads)] for n in server.lens]
    assert server.lens == [len(p) - 1 for p in prompts]
    check_keys(server, origin, keys, errs)
    g = torch.Generator(device="cuda").manual_seed(5)
    taken = evictions = 0
    for _ in range(10):
        before = [len(t) for t in server.text]
        counts = server.step(torch.rand(server.B * server.nodes, generator=g, device="cuda"))
        taken += sum(counts)
        for b, c in enumerate(counts):
            assert len(server.text[b]) == before[b] + c + 1
            for rows in origin[b]:
                rows += range(before[b] - 1, before[b] + c)     # the text's last token and the accepted ones
        if server.kept is not None:
            kept = server.kept.cpu().numpy()
            for b in range(server.B):
                for h in range(server.block.kv_heads):
                    if kept[b, h, 0] >= 0:
                        evictions += 1
                        old = origin[b][h]
                        mine = kept[b, h][kept[b, h] >= 0]
                        assert np.all(np.diff(mine) > 0)
                        assert old[-8:] == [old[i] for i in mine[-8:]] and mine[0] == 0
                        origin[b][h] = [old[i] for i in mine]
        check_keys(server, origin, keys, errs)
    assert moe.get_device_error(server.block.ws) == 0 and moe.get_device_error(server.ws) == 0
    assert taken > 0 and (evictions > 0) == (budget < 200)
    if budget >= 200:
        # every row of the text but the last token's gave its weight of 1 per query head
        table, w = server.table.cpu().numpy(), server.weights.double().cpu().numpy()
        group = server.block.q_heads // server.block.kv_heads
        for b in range(server.B):
            j = np.arange(server.lens[b])
            total = w[table[b, j // page], :, j % page].sum(0)
            rows = server.lens[b]
            assert np.all(np.abs(total - rows * group) <= rows * group * 2.0 ** -14)


def test_a_step_on_another_stream():
    """The operators in turn on a stream of their own give what they give on the current one, also behind
    work that is still queued there when they are called."""
    rng = np.random.default_rng(41)
    batch, heads, page, D = Batch(rng, [(200, 12), (37, 5), (0, 9)], 16), 2, 16, 64
    planes = cache_planes(rng, batch.num_pages + 30, heads, page, D)
    q = activations(rng, (batch.T, heads * 2, D), "bf16").cuda()
    bits = [[(2 << i) - 1 for i in range(n)] for _, n in batch.pairs]
    mask = torch.tensor([[v] for t in bits for v in t], dtype=torch.int32).cuda()
    keep = torch.tensor([[0, 2, 5], [1, 2, 4], [0, 3, 8]], dtype=torch.int32).cuda()
    new_table = torch.arange(batch.num_pages, batch.num_pages + 30, dtype=torch.int32).view(3, 10).cuda()

    def step(stream):
        cache, dev = device_cache(planes), batch.device()
        out, lse = torch.empty_like(q), torch.empty(q.shape[:2], device="cuda")
        weights = torch.rand(batch.num_pages + 30, heads, page, device="cuda", generator=torch.Generator("cuda").manual_seed(2))
        normed = torch.empty_like(q.flatten(1))
        lens, cut = torch.empty(3, dtype=torch.int32, device="cuda"), torch.empty(3, dtype=torch.int32, device="cuda")
        kept, three = torch.empty(3, heads, 40, dtype=torch.int32, device="cuda"), torch.full_like(lens, 3)
        size = max(moe.attention_workspace_bytes(heads * 2, heads, D), moe.kv_keep_workspace_bytes(),
                   moe.kv_weights_workspace_bytes(batch.T, heads * 2, heads, D), moe.kv_evict_workspace_bytes(3, heads))
        spaces = [zeros_ws(size) for _ in range(4)]
        torch.cuda.synchronize()
        if stream is not None:
            with torch.cuda.stream(stream):
                busy = torch.ones(4096, 4096, device="cuda")
                for _ in range(8):
                    busy = busy @ busy * 2.0 ** -12
        moe.moe_attention_tree_e4m3(q, cache, dev, mask, out, spaces[0], lse=lse, stream=stream)
        moe.moe_kv_weights_e4m3(q, lse, cache, dev, weights, spaces[1], decay=0.5, stream=stream)
        moe.moe_residual_norm(out.flatten(1), q.flatten(1), normed=normed, stream=stream)
        moe.moe_kv_keep_e4m3(cache, dev, keep, three, lens, spaces[2], stream=stream)
        after = moe.SeqBatch(dev.q_offsets, lens, dev.page_table)
        moe.moe_kv_evict_e4m3(cache, after, weights, new_table, kept, cut, spaces[3], first=2, recent=7, stream=stream)
        torch.cuda.synchronize()
        assert all(moe.get_device_error(ws) == 0 for ws in spaces)
        return [out, lse, normed, weights, lens, kept, cut, cache.k_codes, cache.v_codes, cache.k_scales, cache.v_scales]

    for a, b in zip(step(None), step(torch.cuda.Stream())):
        assert torch.equal(a, b)


def test_operators_wait_for_their_stream():
    """Work queued on a stream puts the inputs into place, behind long work: operators that are called on that
    stream, while another is the current one, see them, and would see the inputs' old values anywhere else."""
    rng = np.random.default_rng(43)
    batch, heads, page, D = Batch(rng, [(200, 12), (37, 5), (0, 9)], 16), 2, 16, 64
    planes = cache_planes(rng, batch.num_pages + 30, heads, page, D)
    wrong = cache_planes(rng, batch.num_pages + 30, heads, page, D)
    q = activations(rng, (batch.T, heads * 2, D), "bf16").cuda()
    other_q = activations(rng, (batch.T, heads * 2, D), "bf16").cuda()
    mask = torch.tensor([[(2 << i) - 1] for _, n in batch.pairs for i in range(n)], dtype=torch.int32).cuda()
    keep = torch.tensor([[0, 2, 5], [1, 2, 4], [0, 3, 8]], dtype=torch.int32).cuda()
    new_table = torch.arange(batch.num_pages, batch.num_pages + 30, dtype=torch.int32).view(3, 10).cuda()
    w = torch.from_numpy(rng.random((batch.num_pages + 30, heads, page), np.float32)).cuda()
    size = max(moe.attention_workspace_bytes(heads * 2, heads, D), moe.kv_keep_workspace_bytes(),
               moe.kv_weights_workspace_bytes(batch.T, heads * 2, heads, D), moe.kv_evict_workspace_bytes(3, heads))

    def step(stream):
        right, cache, dev = device_cache(planes), device_cache(wrong), batch.device()
        x, weights, list_ = other_q.clone(), torch.zeros_like(w), torch.zeros_like(keep)
        pairs = [(x, q), (weights, w), (list_, keep), (cache.k_codes, right.k_codes), (cache.v_codes, right.v_codes),
                 (cache.k_scales, right.k_scales), (cache.v_scales, right.v_scales)]
        out, lse = torch.empty_like(q), torch.empty(q.shape[:2], device="cuda")
        normed, bits = torch.empty_like(q.flatten(1)), torch.ones_like(mask)
        lens, cut, three = (torch.full((3,), 3, dtype=torch.int32, device="cuda") for _ in range(3))
        kept = torch.empty(3, heads, 40, dtype=torch.int32, device="cuda")
        spaces = [zeros_ws(size) for _ in range(4)]
        busy = torch.ones(8192, 8192, device="cuda")
        torch.cuda.synchronize()
        with torch.cuda.stream(stream):
            for _ in range(4 if stream is not None else 0):
                busy = busy @ busy * 2.0 ** -13
            for to, src in pairs + [(bits, mask)]:
                to.copy_(src)
        moe.moe_attention_tree_e4m3(x, cache, dev, bits, out, spaces[0], lse=lse, stream=stream)
        moe.moe_kv_weights_e4m3(x, lse, cache, dev, weights, spaces[1], decay=0.5, stream=stream)
        moe.moe_residual_norm(out.flatten(1), x.flatten(1), normed=normed, stream=stream)
        moe.moe_kv_keep_e4m3(cache, dev, list_, three, lens, spaces[2], stream=stream)
        after = moe.SeqBatch(dev.q_offsets, lens, dev.page_table)
        moe.moe_kv_evict_e4m3(cache, after, weights, new_table, kept, cut, spaces[3], first=2, recent=7, stream=stream)
        queued = stream is None or not stream.query()            # all of it was called while the stream was busy
        torch.cuda.synchronize()
        assert all(moe.get_device_error(ws) == 0 for ws in spaces)
        return queued, [out, lse, normed, weights, lens, kept, cut, cache.k_codes, cache.v_codes, cache.k_scales,
                        cache.v_scales]

    _, want = step(None)
    queued, got = step(torch.cuda.Stream())
    assert queued
    for a, b in zip(got, want):
        assert torch.equal(a, b)
