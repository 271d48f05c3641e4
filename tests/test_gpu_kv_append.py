"""moe_kv_append_rope_e4m3 against the oracle: codes, scales and rotated queries bit for bit (the
definition is single float32 operations in a fixed order)."""
import numpy as np
import pytest
import torch

import nvfp4_grouped_gemm_gb300 as moe
from oracle import serving as oracle
from serving_util import Batch, activations, cache_planes, device_cache, zeros_ws

pytestmark = pytest.mark.gpu


def tables(max_pos, rotary, rng):
    ang = rng.uniform(0, 2 * np.pi, (max_pos, rotary // 2))
    return np.cos(ang).astype(np.float32), np.sin(ang).astype(np.float32)


def bits(t):
    return t.cpu().view(torch.int16).numpy()


def places_of(batch):
    return np.concatenate([np.arange(n) + p for p, n in batch.pairs]).astype(np.int64)


def check(rng, pairs, page, heads, qh, D, rotary, inter, dtype, amp=1.0, positions=None, in_place=False,
          strided=False, bad_page=None, planes=None, max_pos=None):
    batch = Batch(rng, pairs, page)
    if bad_page is not None:
        batch.table[bad_page] = batch.num_pages + 5
    planes = planes or cache_planes(rng, batch.num_pages, heads, page, D)
    T = batch.T
    k, v, q = (activations(rng, (T, h, D), dtype, amp) for h in (heads, heads, qh))
    max_pos = max_pos or (max(int(batch.lens.max()), 1) + 3)
    cos, sin = tables(max_pos, max(rotary, 2), rng)
    pos = places_of(batch) if positions is None else positions.astype(np.int64)
    at = np.clip(pos, 0, max_pos - 1)
    ref = [p.copy() for p in planes]
    turn = (lambda x: oracle.rotate(x.float().numpy(), cos[at][:, None], sin[at][:, None], inter)) \
        if rotary else (lambda x: x.float().numpy())
    oracle.kv_append(ref[0], ref[1], turn(k), batch.offsets, batch.lens, batch.table)
    oracle.kv_append(ref[2], ref[3], v.float().numpy(), batch.offsets, batch.lens, batch.table)
    want_q = torch.from_numpy(turn(q)).to(q.dtype)

    cache = device_cache(planes)
    if strided:              # q, k, v as slices of one projection's output rows
        rows = torch.cat([x.reshape(T, -1) for x in (q, k, v)], 1).cuda()
        dq, dk, dv = (s.view(T, -1, D) for s in rows.split([qh * D, heads * D, heads * D], 1))
    else:
        dq, dk, dv = q.cuda(), k.cuda(), v.cuda()
    out = dq if in_place else torch.empty(T, qh, D, dtype=q.dtype, device="cuda")
    ws = zeros_ws(moe.kv_append_workspace_bytes())
    moe.moe_kv_append_rope_e4m3(
        cache, batch.device(), dk, dv, torch.from_numpy(cos).cuda() if rotary else None,
        torch.from_numpy(sin).cuda() if rotary else None, ws, q=dq, q_out=out,
        positions=None if positions is None else torch.from_numpy(positions).cuda(),
        interleaved=inter)
    err = moe.get_device_error(ws)
    assert np.array_equal(bits(out.contiguous()), bits(want_q))
    for got, want in zip((cache.k_codes, cache.k_scales, cache.v_codes, cache.v_scales), ref):
        assert np.array_equal(got.cpu().numpy(), want)
    return err


@pytest.mark.parametrize("D,page,heads,qh,rotary,inter,dtype", [
    (128, 64, 8, 32, 128, False, "bf16"), (64, 16, 2, 5, 64, True, "f16"),
    (256, 128, 1, 3, 128, False, "f16"), (128, 32, 3, 7, 48, True, "bf16"),
    (64, 64, 4, 4, 0, False, "bf16"), (128, 16, 1, 1, 16, False, "f16")])
def test_single_tokens_prompts_and_page_edges(D, page, heads, qh, rotary, inter, dtype):
    rng = np.random.default_rng(D + page)
    pairs = [(0, 1), (page - 1, 1), (page, 1), (page - 1, 2), (3, page), (0, 2 * page + 1), (5, 0),
             (0, 0), (page // 2, 3 * page)]
    assert check(rng, pairs, page, heads, qh, D, rotary, inter, dtype) == 0


def test_one_token_of_one_sequence():
    assert check(np.random.default_rng(3), [(1000, 1)], 64, 8, 32, 128, 128, False, "bf16") == 0


def test_more_sequences_than_a_block_has_threads():
    rng = np.random.default_rng(4)
    pairs = [(int(rng.integers(0, 40)), int(rng.integers(0, 3))) for _ in range(700)]
    assert check(rng, pairs, 16, 1, 1, 64, 64, False, "bf16") == 0


@pytest.mark.parametrize("amp", [1e-30, 1e-4, 300.0, 3e37])
def test_magnitudes_from_tiny_to_huge(amp):
    rng = np.random.default_rng(5)
    with np.errstate(over="ignore", invalid="ignore"):
        assert check(rng, [(20, 7), (0, 33)], 32, 2, 2, 64, 64, False, "bf16", amp=amp) == 0


def test_a_zero_page_and_a_scale_that_grows():
    """All-zero values give the smallest scale; a louder later token raises a page's scale and
    the earlier codes follow it (also from a scale that is not a power of two)."""
    rng = np.random.default_rng(6)
    assert check(rng, [(0, 20)], 32, 2, 2, 64, 64, False, "f16", amp=0.0) == 0
    planes = list(cache_planes(rng, 8, 2, 32, 64))
    planes[1][:] = np.float32(2.0 ** -12)
    planes[3][:] = np.float32(0.00071)
    assert check(rng, [(30, 5), (1, 2)], 32, 2, 2, 64, 64, False, "bf16", amp=5.0,
                 planes=tuple(planes)) == 0


def test_token_by_token_keeps_earlier_values():
    """Tokens appended one call at a time, each louder than the last, against the oracle."""
    rng = np.random.default_rng(7)
    P, D, n = 16, 64, 20
    k = (rng.standard_normal((n, 1, D)) * 1.4 ** np.arange(n)[:, None, None]).astype(np.float32)
    kt = torch.from_numpy(k).to(torch.bfloat16)
    codes, scales = np.zeros((2, 1, P, D), np.uint8), np.ones((2, 1), np.float32)
    cache = moe.PagedKvCache.allocate(2, 1, P, D)
    table = np.array([[1, 0]], np.int32)
    ws = zeros_ws(moe.kv_append_workspace_bytes())
    for i in range(n):
        b = moe.SeqBatch(torch.tensor([0, 1], dtype=torch.int32).cuda(),
                         torch.tensor([i + 1], dtype=torch.int32).cuda(), torch.from_numpy(table).cuda())
        row = kt[i:i + 1].cuda()
        moe.moe_kv_append_rope_e4m3(cache, b, row, row, None, None, ws)
        oracle.kv_append(codes, scales, kt[i:i + 1].float().numpy(), [0, 1], [i + 1], table)
    assert np.array_equal(cache.k_codes.cpu().numpy(), codes)
    assert np.array_equal(cache.v_codes.cpu().numpy(), codes)
    assert np.array_equal(cache.k_scales.cpu().numpy(), scales)


def test_rows_of_one_projection_and_in_place_queries():
    rng = np.random.default_rng(8)
    assert check(rng, [(7, 9), (60, 11)], 64, 4, 16, 128, 128, False, "bf16", strided=True) == 0
    assert check(rng, [(7, 9), (60, 11)], 64, 4, 16, 128, 128, True, "bf16", strided=True,
                 in_place=True) == 0


def test_given_positions_and_positions_past_the_table():
    rng = np.random.default_rng(9)
    pos = rng.integers(0, 50, 12).astype(np.int32)
    assert check(rng, [(3, 12)], 16, 1, 2, 64, 64, False, "f16", positions=pos, max_pos=50) == 0
    pos[4], pos[7] = 50, -1
    assert check(rng, [(3, 12)], 16, 1, 2, 64, 64, False, "f16", positions=pos, max_pos=50) == \
        moe.DEVERR_POSITION


def test_bad_pages_and_overlong_sequences_are_left_out_and_reported():
    rng = np.random.default_rng(10)
    assert check(rng, [(0, 40), (5, 3)], 16, 2, 2, 64, 64, False, "bf16", bad_page=(0, 1)) == \
        moe.DEVERR_PAGE
    # a sequence one page longer than its row of the table
    P = 16
    cache = moe.PagedKvCache.allocate(4, 1, P, 64)
    k = activations(rng, (20, 1, 64), "bf16")
    table = np.array([[2]], np.int32)
    codes, scales = np.zeros((4, 1, P, 64), np.uint8), np.ones((4, 1), np.float32)
    oracle.kv_append(codes, scales, k.float().numpy(), [0, 20], [25], table)
    ws = zeros_ws(moe.kv_append_workspace_bytes())
    b = moe.SeqBatch(torch.tensor([0, 20], dtype=torch.int32).cuda(),
                     torch.tensor([25], dtype=torch.int32).cuda(), torch.from_numpy(table).cuda())
    moe.moe_kv_append_rope_e4m3(cache, b, k.cuda(), k.cuda(), None, None, ws)
    assert moe.get_device_error(ws) == moe.DEVERR_PAGE
    assert np.array_equal(cache.k_codes.cpu().numpy(), codes)
    # more new tokens than the sequence is long: the first ones have no place
    b = moe.SeqBatch(torch.tensor([0, 20], dtype=torch.int32).cuda(),
                     torch.tensor([9], dtype=torch.int32).cuda(), torch.from_numpy(table).cuda())
    oracle.kv_append(codes, scales, k.float().numpy(), [0, 20], [9], table)
    moe.moe_kv_append_rope_e4m3(cache, b, k.cuda(), k.cuda(), None, None, ws)
    assert moe.get_device_error(ws) == moe.DEVERR_PAGE
    assert np.array_equal(cache.k_codes.cpu().numpy(), codes)


def test_nan_stays_in_its_own_code():
    rng = np.random.default_rng(11)
    k = activations(rng, (5, 1, 64), "bf16")
    k[2, 0, 7] = float("nan")
    cache = moe.PagedKvCache.allocate(1, 1, 16, 64)
    codes, scales = np.zeros((1, 1, 16, 64), np.uint8), np.ones((1, 1), np.float32)
    clean = k.clone()
    clean[2, 0, 7] = 0
    oracle.kv_append(codes, scales, clean.float().numpy(), [0, 5], [5], np.zeros((1, 1), np.int32))
    codes[0, 0, 2, 7] = 0x7F
    b = moe.SeqBatch(torch.tensor([0, 5], dtype=torch.int32).cuda(),
                     torch.tensor([5], dtype=torch.int32).cuda(), torch.zeros(1, 1, dtype=torch.int32).cuda())
    moe.moe_kv_append_rope_e4m3(cache, b, k.cuda(), k.cuda(), None, None,
                                zeros_ws(moe.kv_append_workspace_bytes()))
    got = cache.v_codes.cpu().numpy()
    got[0, 0, 2, 7] &= 0x7F
    assert np.array_equal(got, codes)
    assert np.array_equal(cache.v_scales.cpu().numpy(), scales)


@pytest.mark.parametrize("D,qh,inter,dtype,pairs", [
    (64, 13, False, "bf16", [(0, 5000), (17, 1203)]),                  # 2, 4 and 8 query heads per thread,
    (128, 7, True, "f16", [(5, 9000), (0, 1), (100, 2203)]),           # the last group short
    (256, 11, False, "bf16", [(0, 7101)])])
def test_many_tokens_with_odd_numbers_of_query_heads(D, qh, inter, dtype, pairs):
    assert check(np.random.default_rng(12), pairs, 128, 1, qh, D, D, inter, dtype) == 0


@pytest.mark.parametrize("length", [0, -1, -(1 << 31), 3 - (1 << 31)])
def test_lengths_below_the_new_tokens_leave_pages_alone(length):
    rng = np.random.default_rng(23)
    cache = moe.PagedKvCache.allocate(4, 1, 16, 64)
    k = activations(rng, (6, 1, 64), "bf16").cuda()
    b = moe.SeqBatch(torch.tensor([0, 6], dtype=torch.int32).cuda(), torch.tensor([length], dtype=torch.int32).cuda(),
                     torch.tensor([[1, 2]], dtype=torch.int32).cuda())
    ws = zeros_ws(moe.kv_append_workspace_bytes())
    moe.moe_kv_append_rope_e4m3(cache, b, k, k, None, None, ws)
    assert moe.get_device_error(ws) == moe.DEVERR_PAGE
    assert not cache.k_codes.any() and not cache.v_codes.any()
    assert torch.all(cache.k_scales == 1) and torch.all(cache.v_scales == 1)
