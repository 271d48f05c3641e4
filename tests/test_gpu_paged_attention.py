"""moe_attention_paged_e4m3 against the float64 oracle, within the oracle's error bound plus the
rounding of the output type."""
import numpy as np
import pytest
import torch

import nvfp4_grouped_gemm_gb300 as moe
from oracle import serving as oracle
from serving_util import Batch, activations, cache_planes, device_cache, zeros_ws

pytestmark = pytest.mark.gpu
# half a unit in the last place of 8 and 11 significant bits, and half the least subnormal
ROUND = {"bf16": (2.0 ** -8, 2.0 ** -134), "f16": (2.0 ** -11, 2.0 ** -25)}


def stale_nan(planes, batch):
    """NaN codes in every slot that no sequence uses."""
    used = np.zeros((batch.num_pages, batch.page), bool)
    for b, n in enumerate(batch.lens):
        for i in range(min(int(n), batch.table.shape[1] * batch.page)):
            if 0 <= batch.table[b, i // batch.page] < batch.num_pages:
                used[batch.table[b, i // batch.page], i % batch.page] = True
    for c in (planes[0], planes[2]):
        c.transpose(0, 2, 1, 3)[~used] = 0x7F


def run(q, cache, batch, qh, D, scale, window=0, ws=None, out=None, stream=None):
    T = q.shape[0]
    out = torch.full((T, qh, D), float("nan"), dtype=q.dtype, device="cuda") if out is None else out
    lse = torch.full((T, qh), float("nan"), device="cuda")
    ws = zeros_ws(moe.attention_workspace_bytes(qh, cache.kv_heads, D)) if ws is None else ws
    moe.moe_attention_paged_e4m3(q, cache, batch, out, ws, scale=scale, window=window, lse=lse,
                                 stream=stream)
    return out, lse, ws


def check(rng, pairs, page, heads, group, D, dtype, window=0, amp=1.0, planes=None, scale=None,
          edit=None, err=0):
    batch = Batch(rng, pairs, page)
    if edit:
        edit(batch)
    planes = planes(batch) if planes else cache_planes(rng, batch.num_pages, heads, page, D)
    stale_nan(planes, batch)
    q = activations(rng, (batch.T, heads * group, D), dtype, amp)
    scale = D ** -0.5 if scale is None else scale
    want, wl, eo, el = oracle.attention(q.double().numpy(), *planes, batch.offsets, batch.lens,
                                        batch.table, scale, window)
    out, lse, ws = run(q.cuda(), device_cache(planes), batch.device(), heads * group, D, scale, window)
    assert moe.get_device_error(ws) == err
    got, gl = out.double().cpu().numpy(), lse.double().cpu().numpy()
    rel, floor = ROUND[dtype]
    tol = eo + rel * (np.abs(want) + eo) + floor
    assert np.all(np.abs(got - want) <= tol), float(np.max(np.abs(got - want) / tol))
    seen = np.isfinite(wl)
    assert np.array_equal(np.isfinite(gl), seen) and np.all(gl[~seen] == -np.inf)
    assert np.all(np.abs(gl[seen] - wl[seen]) <= el[seen] + 1e-6)
    assert np.all(got[~seen] == 0)
    return out, lse


@pytest.mark.parametrize("D,page,heads,group,dtype", [
    (128, 64, 2, 4, "bf16"), (64, 16, 1, 1, "f16"), (128, 16, 1, 8, "f16"), (256, 32, 1, 5, "bf16"),
    (64, 128, 2, 16, "bf16"), (128, 128, 1, 12, "bf16"), (256, 16, 2, 2, "f16"), (64, 64, 1, 33, "f16")])
def test_single_tokens_over_ragged_lengths(D, page, heads, group, dtype):
    rng = np.random.default_rng(D + page + group)
    pairs = [(n - 1, 1) for n in (1, 2, page - 1, page, page + 1, 7 * page + 5, 300, 1025)] + [(40, 0), (0, 0)]
    check(rng, pairs, page, heads, group, D, dtype)


@pytest.mark.parametrize("D,page,heads,group,dtype,pairs", [
    (128, 64, 2, 4, "bf16", [(100, 8), (0, 3), (511, 5), (64, 16)]),
    (64, 16, 1, 5, "f16", [(0, 1), (0, 17), (33, 31), (700, 4)]),
    (256, 32, 1, 2, "bf16", [(10, 40), (200, 9)]),
    (128, 16, 1, 1, "bf16", [(5, 130)]),
    (128, 64, 1, 4, "bf16", [(0, 129), (300, 64), (3, 1)]),
    (64, 64, 2, 8, "f16", [(77, 100), (0, 200)]),
    (128, 128, 1, 7, "f16", [(1000, 37), (0, 150)])])
def test_several_new_tokens_are_causal(D, page, heads, group, dtype, pairs):
    check(np.random.default_rng(group + D), pairs, page, heads, group, D, dtype)


@pytest.mark.parametrize("window", [1, 7, 64, 100])
def test_windows(window):
    rng = np.random.default_rng(window)
    check(rng, [(0, 1), (500, 1), (63, 30), (200, 70)], 64, 2, 4, 128, "bf16", window=window)
    check(rng, [(0, 5), (130, 160)], 16, 1, 2, 64, "f16", window=window)


def test_a_long_sequence_beside_short_ones():
    rng = np.random.default_rng(21)
    check(rng, [(20000, 1), (3, 1), (0, 1), (4095, 1)], 64, 1, 8, 128, "bf16")


def test_rows_that_see_nothing():
    """More new tokens than the sequence is long: the first rows have no place and see nothing."""
    rng = np.random.default_rng(22)

    def edit(b):
        b.lens[0], b.lens[1] = 3, 0
    check(rng, [(0, 9), (0, 4), (8, 2)], 16, 2, 3, 64, "bf16", edit=edit, err=moe.DEVERR_PAGE)


def test_sharp_and_flat_scores():
    rng = np.random.default_rng(23)
    check(rng, [(900, 4)], 32, 1, 4, 128, "bf16", amp=40.0)
    check(rng, [(900, 4)], 32, 1, 4, 128, "f16", amp=0.0)


def test_large_and_small_activations():
    rng = np.random.default_rng(24)
    check(rng, [(90, 2)], 16, 1, 2, 64, "bf16", amp=1e20, scale=1e-21)
    check(rng, [(90, 2)], 16, 1, 2, 64, "bf16", amp=1e-20, scale=1e18)


def test_pages_whose_scales_lie_far_apart():
    """Value scales from 2^-40 to 2^40 and zero pages with the smallest scale an append writes."""
    rng = np.random.default_rng(25)

    def planes(batch):
        p = list(cache_planes(rng, batch.num_pages, 2, 16, 64))
        p[3] = (2.0 ** rng.integers(-40, 41, p[3].shape)).astype(np.float32)
        p[1] = (rng.uniform(0.5, 2, p[1].shape) * 0.003).astype(np.float32)
        p[2][::3] = 0
        p[3][::3] = np.float32(2.0 ** -64)
        return tuple(p)
    check(rng, [(700, 3), (80, 1)], 16, 2, 4, 64, "bf16", planes=planes)


def test_bad_pages_are_left_out_and_reported():
    rng = np.random.default_rng(26)

    def edit(b):
        b.table[0, 2], b.table[1, 0] = -1, b.num_pages
    check(rng, [(100, 2), (10, 1), (40, 3)], 16, 2, 2, 128, "bf16", edit=edit, err=moe.DEVERR_PAGE)


def test_a_sequence_longer_than_its_table():
    rng = np.random.default_rng(27)

    def edit(b):
        b.lens[0] = b.table.shape[1] * b.page + 9
        b.table[0] = np.arange(b.table.shape[1]) % b.num_pages
    check(rng, [(60, 2), (4, 1)], 16, 1, 2, 64, "bf16", edit=edit, err=moe.DEVERR_PAGE)


def test_pages_spaced_past_32_bits():
    """Pages more than 2^31 bytes apart in one allocation."""
    rng = np.random.default_rng(28)
    heads, P, D = 1, 16, 64
    batch = Batch(rng, [(40, 1)], P, spare=0)
    planes = cache_planes(rng, batch.num_pages, heads, P, D)
    stride = (1 << 31) + 4096
    big = torch.zeros(2 * P * D + stride * (batch.num_pages - 1), dtype=torch.uint8, device="cuda")
    shape, st = (batch.num_pages, heads, P, D), (stride, P * D, D, 1)
    k, v = big.as_strided(shape, st), big.as_strided(shape, st, P * D)
    k.copy_(torch.from_numpy(planes[0]).cuda())
    v.copy_(torch.from_numpy(planes[2]).cuda())
    cache = moe.PagedKvCache(k, v, torch.from_numpy(planes[1]).cuda(), torch.from_numpy(planes[3]).cuda())
    q = activations(rng, (1, 4, D), "bf16").cuda()
    a = run(q, cache, batch.device(), 4, D, 0.125)
    b = run(q, device_cache(planes), batch.device(), 4, D, 0.125)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_strided_queries_outputs_and_no_lse():
    rng = np.random.default_rng(29)
    batch = Batch(rng, [(100, 3), (30, 2)], 64)
    planes = cache_planes(rng, batch.num_pages, 2, 64, 128)
    cache = device_cache(planes)
    rows = activations(rng, (batch.T, 12 * 128), "bf16").cuda()
    q = rows[:, :8 * 128].view(batch.T, 8, 128)
    a, _, _ = run(q.contiguous(), cache, batch.device(), 8, 128, 0.1)
    wide = torch.zeros(batch.T, 12, 128, dtype=torch.bfloat16, device="cuda")
    ws = zeros_ws(moe.attention_workspace_bytes(8, 2, 128))
    moe.moe_attention_paged_e4m3(q, cache, batch.device(), wide[:, 2:10], ws, scale=0.1)
    assert torch.equal(wide[:, 2:10], a)
    assert not wide[:, :2].any() and not wide[:, 10:].any()


def test_repeated_calls_graph_replays_and_another_stream_agree():
    """The same workspace serves call after call, in a graph whose lengths change between
    replays, and the results are the same bits."""
    rng = np.random.default_rng(30)
    pairs = [(3000, 1), (64, 1), (0, 1), (777, 1)]
    batch = Batch(rng, pairs, 32)
    cache = device_cache(cache_planes(rng, batch.num_pages, 2, 32, 128))
    dev = batch.device()
    q = activations(rng, (4, 16, 128), "bf16").cuda()
    a, la, ws = run(q, cache, dev, 16, 128, 0.09)
    for _ in range(3):
        b, lb, _ = run(q, cache, dev, 16, 128, 0.09, ws=ws)
        assert torch.equal(a, b) and torch.equal(la, lb)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        c, lc, _ = run(q, cache, dev, 16, 128, 0.09, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(a, c) and torch.equal(la, lc)
    out, lse = torch.empty_like(a), torch.empty_like(la)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        moe.moe_attention_paged_e4m3(q, cache, dev, out, ws, scale=0.09, lse=lse)
    graph.replay()
    assert torch.equal(a, out)
    dev.seq_lens.copy_(torch.tensor([1500, 10, 1, 778], dtype=torch.int32))
    graph.replay()
    d, ld, _ = run(q, cache, dev, 16, 128, 0.09)
    assert torch.equal(d, out) and torch.equal(ld, lse)
    assert moe.get_device_error(ws) == 0


# ---- sequences of many rows (the tensor-memory form), alone and beside short ones ----
@pytest.mark.parametrize("D,page,heads,group,dtype,pairs", [
    (128, 64, 1, 4, "bf16", [(5000, 70), (0, 300)]),
    (64, 32, 2, 4, "f16", [(0, 512), (1000, 12), (3, 1)]),
    (128, 16, 2, 1, "bf16", [(129, 257), (40, 2), (0, 48), (0, 47)]),
    (128, 128, 1, 3, "f16", [(255, 171)]),
    (64, 16, 1, 16, "bf16", [(2000, 3), (2000, 8), (0, 33)]),
    (128, 64, 3, 8, "bf16", [(64, 6), (1000, 6), (0, 6), (127, 7)])])
def test_many_rows_per_sequence(D, page, heads, group, dtype, pairs):
    check(np.random.default_rng(D + group), pairs, page, heads, group, D, dtype)


def test_many_rows_that_see_nothing():
    rng = np.random.default_rng(31)

    def edit(b):
        b.lens[0], b.lens[2] = 20, 0
    check(rng, [(0, 90), (30, 80), (0, 70)], 16, 1, 2, 64, "bf16", edit=edit, err=moe.DEVERR_PAGE)


def test_many_rows_over_bad_pages_far_scales_and_sharp_scores():
    rng = np.random.default_rng(32)

    def edit(b):
        b.table[0, 1], b.table[0, 9] = -1, b.num_pages
    check(rng, [(100, 80)], 16, 2, 2, 128, "bf16", edit=edit, err=moe.DEVERR_PAGE)

    def planes(batch):
        p = list(cache_planes(rng, batch.num_pages, 1, 16, 64))
        p[3] = (2.0 ** rng.integers(-40, 41, p[3].shape)).astype(np.float32)
        p[2][::3] = 0
        p[3][::3] = np.float32(2.0 ** -64)
        return tuple(p)
    check(rng, [(300, 100)], 16, 1, 3, 64, "bf16", planes=planes)
    check(rng, [(300, 100)], 64, 1, 2, 128, "bf16", amp=40.0)
    check(rng, [(300, 100)], 64, 1, 2, 128, "f16", amp=0.0)
    check(rng, [(90, 60)], 16, 1, 2, 64, "bf16", amp=1e20, scale=1e-21)


def test_many_rows_repeat_bit_for_bit_and_in_graphs():
    rng = np.random.default_rng(33)
    batch = Batch(rng, [(700, 200), (90, 1), (0, 400)], 64)
    cache = device_cache(cache_planes(rng, batch.num_pages, 2, 64, 128))
    dev = batch.device()
    q = activations(rng, (batch.T, 8, 128), "bf16").cuda()
    a, la, ws = run(q, cache, dev, 8, 128, 0.09)
    for _ in range(3):
        b, lb, _ = run(q, cache, dev, 8, 128, 0.09, ws=ws)
        assert torch.equal(a, b) and torch.equal(la, lb)
    out, lse = torch.empty_like(a), torch.empty_like(la)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        moe.moe_attention_paged_e4m3(q, cache, dev, out, ws, scale=0.09, lse=lse)
    for _ in range(2):
        graph.replay()
        assert torch.equal(a, out) and torch.equal(la, lse)
    assert moe.get_device_error(ws) == 0


def test_nan_and_infinite_queries_stay_in_their_rows():
    rng = np.random.default_rng(34)
    for pairs in ([(100, 1), (40, 1)], [(100, 60), (40, 1)]):
        batch = Batch(rng, pairs, 16)
        cache = device_cache(cache_planes(rng, batch.num_pages, 1, 16, 64))
        q = activations(rng, (batch.T, 2, 64), "bf16")
        a, la, _ = run(q.cuda(), cache, batch.device(), 2, 64, 0.1)
        q[0, 1, 3] = float("nan")
        b, lb, _ = run(q.cuda(), cache, batch.device(), 2, 64, 0.1)
        assert torch.isnan(b[0, 1]).all() and torch.isnan(lb[0, 1])
        keep = torch.ones(batch.T, 2, dtype=torch.bool)
        keep[0, 1] = False
        assert torch.equal(a[keep.cuda()], b[keep.cuda()]) and torch.equal(la[keep.cuda()], lb[keep.cuda()])


def test_more_sequences_than_a_block_has_threads():
    rng = np.random.default_rng(35)
    pairs = [(int(rng.integers(0, 40)), int(rng.choice([0, 1, 2, 9, 10, 17]))) for _ in range(1400)]
    check(rng, pairs, 16, 1, 8, 64, "bf16")


@pytest.mark.parametrize("window", [0, 50])
def test_more_blocks_of_rows_than_a_warp_has_lanes(window):
    check(np.random.default_rng(36), [(0, 300), (37, 280), (5, 1)], 16, 1, 33, 64, "f16", window=window)


def test_many_rows_whose_largest_score_comes_late():
    rng = np.random.default_rng(37)
    check(rng, [(2500, 80)], 64, 1, 2, 128, "bf16", amp=40.0)

    def planes(batch):                           # every page's keys four times the one's before
        p = list(cache_planes(rng, batch.num_pages, 1, 64, 64))
        for i, page in enumerate(batch.table[0][:20]):
            p[1][page] = np.float32(2.0 ** (2 * i - 30))
        return tuple(p)
    check(rng, [(1100, 90)], 64, 1, 2, 64, "f16", planes=planes)


# ---- factors of the scores below the least float32 ----
@pytest.mark.parametrize("window", [0, 40])
@pytest.mark.parametrize("pairs", [[(100, 3), (20, 1)], [(100, 90), (0, 140), (7, 2)]])
def test_tiny_queries_and_zero_keys_hide_what_a_row_does_not_see(pairs, window):
    """scale * k_scale times a row's power of two may underflow to 0; hidden keys stay hidden."""
    rng = np.random.default_rng(38)
    check(rng, pairs, 16, 1, 2, 64, "bf16", window=window, amp=2.0 ** -130)

    def planes(batch):                           # the scale that an append gives zero keys
        p = list(cache_planes(rng, batch.num_pages, 2, 64, 128))
        p[0][:], p[1][:] = 0, np.float32(2.0 ** -64)
        return tuple(p)
    check(rng, pairs, 64, 2, 2, 128, "bf16", window=window, amp=2.0 ** -72, planes=planes)
    check(rng, pairs, 64, 2, 2, 128, "bf16", window=window, amp=0.0, planes=planes)


# ---- NaN values that only some rows see ----
@pytest.mark.parametrize("D,page,heads,group,dtype,pairs,window", [
    (128, 64, 2, 4, "bf16", [(100, 1), (63, 1), (500, 1)], 50),         # one token, before its window
    (64, 16, 1, 1, "f16", [(100, 7), (0, 5)], 0),                       # one, two, three row tiles
    (128, 32, 1, 3, "bf16", [(100, 5), (31, 4)], 0),
    (64, 64, 2, 4, "bf16", [(200, 6), (63, 5)], 9),
    (256, 32, 1, 2, "f16", [(70, 6), (0, 9)], 0),
    (256, 16, 1, 1, "bf16", [(70, 3), (0, 9)], 20),
    (128, 64, 1, 2, "bf16", [(300, 100), (0, 150), (64, 3)], 0),        # many rows, and few beside them
    (64, 16, 1, 3, "f16", [(130, 90)], 0),
    (64, 32, 2, 4, "bf16", [(400, 300), (10, 20)], 70),
    (128, 128, 1, 1, "f16", [(1000, 300)], 129)])
def test_nan_values_reach_only_the_rows_that_see_them(D, page, heads, group, dtype, pairs, window):
    """V codes of NaN at places that some new tokens see and others do not (later ones, or before
    the window): those who see the key have NaN in that value, all else is as if the code were 0."""
    rng = np.random.default_rng(39)
    batch = Batch(rng, pairs, page)
    planes = cache_planes(rng, batch.num_pages, heads, page, D)
    stale_nan(planes, batch)
    nan = np.zeros((batch.T, heads * group, D), bool)
    bad = planes[2].copy()
    for b, (past, n) in enumerate(pairs):
        end = past + n
        places = {end - 1, past + n // 2, past}
        if window:                               # just outside and inside some rows' windows
            places |= {p for p in (past - window, past - window + 1, end - 1 - window) if p >= 0}
        for at in places:
            for d, h in ((int(rng.integers(D)), int(rng.integers(heads))), (D - 1, 0), (0, heads - 1)):
                slot = batch.table[b, at // page], h, at % page, d
                planes[2][slot], bad[slot] = 0, int(rng.choice([0x7F, 0xFF]))
                for i in range(n):
                    if at <= past + i and (window == 0 or at > past + i - window):
                        nan[batch.offsets[b] + i, h * group:(h + 1) * group, d] = True
    q = activations(rng, (batch.T, heads * group, D), dtype)
    want, wl, eo, el = oracle.attention(q.double().numpy(), *planes, batch.offsets, batch.lens,
                                        batch.table, D ** -0.5, window)
    clean, cl, _ = run(q.cuda(), device_cache(planes), batch.device(), heads * group, D, D ** -0.5, window)
    planes = planes[:2] + (bad,) + planes[3:]
    out, lse, ws = run(q.cuda(), device_cache(planes), batch.device(), heads * group, D, D ** -0.5, window)
    assert moe.get_device_error(ws) == 0
    assert np.array_equal(torch.isnan(out).cpu().numpy(), nan)
    keep = torch.from_numpy(~nan).cuda()
    assert torch.equal(out[keep], clean[keep]) and torch.equal(lse, cl)
    got = clean.double().cpu().numpy()
    rel, floor = ROUND[dtype]
    assert np.all(np.abs(got - want) <= eo + rel * (np.abs(want) + eo) + floor)
    assert np.all(np.abs(cl.double().cpu().numpy() - wl) <= el + 1e-6)


# ---- value scales further apart than float32's exponents ----
@pytest.mark.parametrize("order", ["mixed", "rising", "falling", "by_fours"])
@pytest.mark.parametrize("D,page,heads,group,pairs", [
    (64, 16, 2, 4, [(700, 3), (80, 1)]), (128, 32, 1, 8, [(6000, 1), (300, 1)]),
    (256, 16, 1, 2, [(500, 3), (90, 1)]), (64, 16, 1, 3, [(300, 100)]),
    (128, 64, 1, 2, [(3000, 90), (400, 1)])])
def test_quiet_values_keep_their_share_of_the_sum(D, page, heads, group, pairs, order):
    """Pages of zeros (scale 2^-64) and quiet ones beside pages near the largest scale an append
    writes: the softmax's sum is over all keys alike, whatever their values' scale."""
    rng = np.random.default_rng(40)
    batch = Batch(rng, pairs, page)
    planes = list(cache_planes(rng, batch.num_pages, heads, page, D))
    for row in batch.table:
        for i, number in enumerate(row[row >= 0]):
            loud = {"mixed": rng.random() < 0.4, "rising": i >= 3, "falling": i < 3,
                    "by_fours": i % 4 < 2}[order]
            planes[3][number] = np.float32(2.0 ** (rng.integers(95, 105) if loud else -64))
            if not loud and rng.random() < 0.5:
                planes[2][number] = 0
    stale_nan(planes, batch)
    for amp in (1.0, 8.0):
        q = activations(rng, (batch.T, heads * group, D), "bf16", amp)
        want, wl, eo, el = oracle.attention(q.double().numpy(), *planes, batch.offsets, batch.lens,
                                            batch.table, D ** -0.5)
        out, lse, ws = run(q.cuda(), device_cache(planes), batch.device(), heads * group, D, D ** -0.5)
        assert moe.get_device_error(ws) == 0
        got, gl = out.double().cpu().numpy(), lse.double().cpu().numpy()
        rel, floor = ROUND["bf16"]
        # the exponents here reach 2^8, where float32 rounds by 2^-17: three times, in natural logarithms
        # less than 2^-16 beside the bound for scores alone; the values' weights have it twice
        eo = eo + 2.0 ** -15 * np.abs(want)
        tol = eo + rel * (np.abs(want) + eo) + floor
        assert np.all(np.abs(got - want) <= tol), float(np.max(np.abs(got - want) / tol))
        assert np.all(np.abs(gl - wl) <= el + 1e-6 + 2.0 ** -16), float(np.max(np.abs(gl - wl)))


# ---- forms that large batches and long sequences run ----
@pytest.mark.parametrize("D,page,heads,group,dtype", [
    (128, 64, 8, 4, "bf16"), (64, 16, 4, 8, "f16"), (256, 32, 4, 2, "bf16"), (128, 16, 3, 1, "f16")])
def test_one_token_of_many_sequences(D, page, heads, group, dtype):
    """More segments (sequences times key heads) than there are SMs, one row tile each."""
    rng = np.random.default_rng(41)
    pairs = [(int(n), 1) for n in np.exp(rng.uniform(0, np.log(700), 64)).astype(int)] + [(0, 0), (3000, 1)]
    check(rng, pairs, page, heads, group, D, dtype)
    check(rng, pairs, page, heads, group, D, dtype, window=37)


@pytest.mark.parametrize("D,n", [(128, 30011), (256, 14003), (64, 40000)])
def test_one_sequence_in_more_pieces_than_a_warp_has_lanes(D, n):
    check(np.random.default_rng(42), [(n, 1)], 64, 1, 2, D, "bf16")


@pytest.mark.parametrize("D,page,window", [(128, 64, 50), (64, 16, 9), (256, 32, 70)])
def test_nan_values_in_many_sequences(D, page, window):
    pairs = [(int(n), 1) for n in np.linspace(0, 400, 60)]
    test_nan_values_reach_only_the_rows_that_see_them(D, page, 4, 2, "bf16", pairs, window)


@pytest.mark.parametrize("order", ["mixed", "rising", "falling"])
def test_quiet_values_in_long_and_in_many_sequences(order):
    test_quiet_values_keep_their_share_of_the_sum(128, 64, 1, 2, [(30011, 1)], order)
    test_quiet_values_keep_their_share_of_the_sum(64, 16, 4, 2, [(int(n), 1) for n in np.linspace(0, 400, 60)], order)


@pytest.mark.parametrize("D,page,heads,group,dtype,pairs,window", [
    (128, 64, 2, 4, "bf16", [(100, 1), (63, 1), (500, 3)], 50), (64, 16, 1, 3, "f16", [(100, 7), (0, 5)], 0),
    (256, 32, 1, 2, "bf16", [(70, 6), (0, 9)], 20), (128, 64, 1, 2, "bf16", [(300, 100), (64, 3)], 0),
    (64, 32, 2, 4, "f16", [(400, 300), (10, 20)], 70)])
def test_nan_keys_reach_only_the_rows_that_see_them(D, page, heads, group, dtype, pairs, window):
    """K codes of NaN at the last new token and before some rows' windows: rows that see the key are
    NaN, the others within their bounds."""
    rng = np.random.default_rng(43)
    batch = Batch(rng, pairs, page)
    planes = cache_planes(rng, batch.num_pages, heads, page, D)
    stale_nan(planes, batch)
    nan = np.zeros((batch.T, heads * group), bool)
    for b, (past, n) in enumerate(pairs):
        for at in {past + n - 1} | ({past + n - 1 - window, past - window} if window else set()):
            if at < 0:
                continue
            h = int(rng.integers(heads))
            planes[0][batch.table[b, at // page], h, at % page, int(rng.integers(D))] = 0x7F
            for i in range(n):
                if at <= past + i and (window == 0 or at > past + i - window):
                    nan[batch.offsets[b] + i, h * group:(h + 1) * group] = True
    q = activations(rng, (batch.T, heads * group, D), dtype)
    want, wl, eo, el = oracle.attention(q.double().numpy(), *planes, batch.offsets, batch.lens,
                                        batch.table, D ** -0.5, window)
    out, lse, ws = run(q.cuda(), device_cache(planes), batch.device(), heads * group, D, D ** -0.5, window)
    assert moe.get_device_error(ws) == 0
    got, gl = out.double().cpu().numpy(), lse.double().cpu().numpy()
    assert np.array_equal(np.isnan(got), np.broadcast_to(nan[:, :, None], got.shape))
    assert np.array_equal(np.isnan(gl), nan) and nan.any() and not nan.all()
    rel, floor = ROUND[dtype]
    tol = eo + rel * (np.abs(want) + eo) + floor
    assert np.all(np.abs(got - want)[~nan] <= tol[~nan])
    assert np.all(np.abs(gl - wl)[~nan] <= el[~nan] + 1e-6)


@pytest.mark.parametrize("length", [-1, -(1 << 31), 3 - (1 << 31)])
@pytest.mark.parametrize("window", [0, 20])
def test_lengths_below_the_new_tokens(length, window):
    rng = np.random.default_rng(77)

    def edit(b):
        b.lens[1] = length
    for group in (2, 20):
        check(rng, [(100, 6), (30, 6), (7, 2)], 16, 2, group, 64, "bf16", window=window, edit=edit, err=moe.DEVERR_PAGE)
