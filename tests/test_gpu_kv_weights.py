"""moe_kv_weights_e4m3 against the float64 oracle, within its error bound."""
import numpy as np
import pytest
import torch

import nvfp4_grouped_gemm_gb300 as moe
from oracle import serving as oracle
from serving_util import Batch, activations, cache_planes, device_cache, zeros_ws

pytestmark = pytest.mark.gpu


def setup(rng, pairs, page, heads, group, D, dtype, window=0, amp=1.0, edit=None, edit_planes=None):
    batch = Batch(rng, pairs, page)
    if edit:
        edit(batch)
    planes = cache_planes(rng, batch.num_pages, heads, page, D)
    q = activations(rng, (batch.T, heads * group, D), dtype, amp)
    lse = oracle.attention(q.double().numpy(), *planes, batch.offsets, batch.lens, batch.table, D ** -0.5,
                           window)[1].astype(np.float32)
    if edit_planes:                                             # behind the attention that left lse
        edit_planes(planes, batch)
    w = (rng.standard_normal((batch.num_pages, heads, page)) ** 2).astype(np.float32)
    return batch, planes, q, lse, w


def call(batch, planes, q, lse, w, window, decay, out=None, cache=None):
    cache = cache or device_cache(planes)
    ws = zeros_ws(moe.kv_weights_workspace_bytes(batch.T, q.shape[1], cache.kv_heads, cache.head_dim))
    weights = torch.from_numpy(w).cuda()
    moe.moe_kv_weights_e4m3(q.cuda(), torch.from_numpy(lse).cuda(), cache, batch.device(), weights, ws,
                            window=window, decay=decay, out=out)
    return (weights if out is None else out), ws


def check(rng, pairs, page, heads, group, D, dtype, window=0, decay=1.0, amp=1.0, edit=None, edit_planes=None, err=0):
    batch, planes, q, lse, w = setup(rng, pairs, page, heads, group, D, dtype, window, amp, edit, edit_planes)
    want, bound = oracle.kv_weights(q.double().numpy(), lse.astype(np.float64), w, planes[0], planes[1],
                                    batch.offsets, batch.lens, batch.table, D ** -0.5, window, decay)
    got, ws = call(batch, planes, q, lse, w, window, decay)
    assert moe.get_device_error(ws) == err
    got = got.cpu().numpy()
    changed = ~(bound == 0)
    assert np.array_equal(got[~changed], w[~changed], equal_nan=True)      # nobody else's slots
    off = np.abs(got.astype(np.float64) - want)
    ok = (off <= bound) | (np.isnan(got) & np.isnan(want))
    assert ok.all(), float(np.nanmax(off[~ok] / bound[~ok]))
    return batch, got


@pytest.mark.parametrize("D,page,heads,group,dtype", [
    (128, 64, 2, 4, "bf16"), (64, 16, 1, 1, "f16"), (128, 16, 1, 8, "f16"), (256, 32, 1, 5, "bf16"),
    (64, 128, 2, 16, "bf16"), (128, 128, 1, 12, "bf16"), (256, 16, 2, 2, "f16"), (64, 64, 1, 33, "f16")])
def test_single_tokens_over_ragged_lengths(D, page, heads, group, dtype):
    rng = np.random.default_rng(D + page + group)
    pairs = [(n - 1, 1) for n in (1, 2, page - 1, page, page + 1, 7 * page + 5, 300, 1025)] + [(40, 0), (0, 0)]
    check(rng, pairs, page, heads, group, D, dtype, decay=0.75)


@pytest.mark.parametrize("D,page,heads,group,dtype,pairs", [
    (128, 64, 2, 4, "bf16", [(100, 8), (0, 3), (511, 5), (64, 16)]),
    (64, 16, 1, 5, "f16", [(0, 1), (0, 17), (33, 31), (700, 4)]),
    (256, 32, 1, 2, "bf16", [(10, 40), (200, 9)]),
    (128, 16, 1, 1, "bf16", [(5, 130)]),
    (128, 64, 1, 7, "f16", [(0, 129), (300, 64), (3, 1)]),
    (64, 64, 2, 3, "bf16", [(77, 100), (0, 45), (1, 0), (9, 2)]),
    (64, 16, 1, 9, "f16", [(60, 61), (300, 29), (1300, 143), (5, 28)])])
def test_several_new_tokens_are_causal(D, page, heads, group, dtype, pairs):
    check(np.random.default_rng(group + D), pairs, page, heads, group, D, dtype)


@pytest.mark.parametrize("window", [1, 7, 64, 100])
def test_windows(window):
    rng = np.random.default_rng(window)
    check(rng, [(0, 1), (500, 1), (63, 30), (200, 70)], 64, 2, 4, 128, "bf16", window=window, decay=0.5)
    check(rng, [(0, 5), (130, 160)], 16, 1, 2, 64, "f16", window=window)


def test_more_rows_than_a_tile_among_single_tokens():
    """As many tokens as sequences, so that the sizes promise single tokens, but one has them all."""
    rng = np.random.default_rng(11)
    check(rng, [(90, 9), (5, 0), (0, 0), (40, 0), (7, 0), (33, 0), (12, 0), (70, 0), (2, 0)], 16, 2, 5, 128, "bf16")
    check(rng, [(90, 3), (40, 0), (5, 0)], 16, 1, 7, 64, "f16")


def test_decay_zero_reads_nothing():
    rng = np.random.default_rng(12)
    batch, planes, q, lse, w = setup(rng, [(130, 2), (50, 9)], 32, 2, 4, 64, "bf16")
    want = call(batch, planes, q, lse, w, 0, 0.0)[0].cpu().numpy()
    used = np.zeros(w.shape, bool)
    for b, n in enumerate(batch.lens):
        for j in range(n):
            used[batch.table[b, j // 32], :, j % 32] = True
    bad = np.where(used, np.float32(np.nan), w)
    got = call(batch, planes, q, lse, bad, 0, 0.0)[0].cpu().numpy()
    assert np.array_equal(got, want)
    check(rng, [(130, 2), (50, 9)], 32, 2, 4, 64, "bf16", decay=0.0)


def test_another_buffer_and_repeated_calls_agree():
    rng = np.random.default_rng(13)
    batch, planes, q, lse, w = setup(rng, [(3000, 3), (77, 1), (600, 20)], 64, 2, 4, 128, "bf16")
    out = torch.full(w.shape, -5.0, device="cuda")
    a = call(batch, planes, q, lse, w, 0, 0.5)[0]
    b = call(batch, planes, q, lse, w, 0, 0.5, out=out)[0]
    touched = b != -5.0
    assert torch.equal(a[touched], b[touched])
    assert int(touched.sum()) == int(batch.lens.sum()) * 2


def test_rows_sum_to_their_number():
    """All rows' weights sum to one each, so the new sums are the number of rows."""
    rng = np.random.default_rng(14)
    batch, planes, q, lse, w = setup(rng, [(700, 5)], 16, 2, 3, 64, "f16")
    got = call(batch, planes, q, lse, w, 0, 0.0)[0].double()
    mine = sum(float(got[batch.table[0, j // 16], :, j % 16].sum()) for j in range(705))
    assert abs(mine - 5 * 6) < 30 * 2.0 ** -16


def test_nan_keys_bad_pages_and_rows_that_saw_nothing():
    rng = np.random.default_rng(15)

    def nan_keys(planes, batch):
        planes[0][batch.table[0, 1], 0, 3, 7] = 0x7F            # token 19 of head 0
        planes[0][batch.table[0, 6], 1, 4, 0] = 0xFF            # a new token, seen from its place on
    _, got = check(rng, [(97, 6), (20, 1)], 16, 2, 3, 64, "bf16", edit_planes=nan_keys)

    def edit(b):
        b.table[0, 2], b.table[1, 0] = -1, b.num_pages
    check(rng, [(100, 2), (10, 1), (40, 3)], 16, 2, 2, 128, "bf16", edit=edit, err=moe.DEVERR_PAGE)

    def short(b):                                               # more new tokens than tokens
        b.lens[0], b.lens[1] = 3, 0
    check(rng, [(0, 9), (0, 4), (8, 2)], 16, 2, 3, 64, "bf16", edit=short, err=moe.DEVERR_PAGE)


def test_stale_slots_and_many_sequences():
    rng = np.random.default_rng(16)
    check(rng, [(int(rng.integers(0, 60)), int(rng.integers(0, 3))) for _ in range(700)], 16, 1, 2, 64, "f16")


def test_offsets_past_32_bits():
    """Pages spaced so that the cache's last pages lie more than 4 GiB in."""
    rng = np.random.default_rng(17)
    batch, planes, q, lse, w = setup(rng, [(200, 2)], 16, 1, 2, 64, "bf16")
    n, stride = batch.num_pages, (5 << 30) // batch.num_pages // 16 * 16
    big = torch.empty(n * stride, dtype=torch.uint8, device="cuda")
    view = torch.as_strided(big, (n, 1, 16, 64), (stride, 16 * 64, 64, 1))
    view.copy_(torch.from_numpy(planes[0]))
    ones = torch.ones(n, 1, device="cuda")
    cache = moe.PagedKvCache(view, view, torch.from_numpy(planes[1]).cuda(), ones)
    want = call(batch, planes, q, lse, w, 0, 1.0)[0]
    assert torch.equal(call(batch, planes, q, lse, w, 0, 1.0, cache=cache)[0], want)


def test_a_graph_with_other_lengths():
    rng = np.random.default_rng(18)
    batch, planes, q, lse, w = setup(rng, [(300, 1), (40, 1)], 16, 2, 4, 128, "bf16")
    cache, dev = device_cache(planes), batch.device()
    ws = zeros_ws(moe.kv_weights_workspace_bytes(2, 8, 2, 128))
    qd, ld, wd = q.cuda(), torch.from_numpy(lse).cuda(), torch.from_numpy(w).cuda()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        moe.moe_kv_weights_e4m3(qd, ld, cache, dev, wd, ws)
    lens = np.array([200, 41], np.int32)                        # shorter than when captured
    dev.seq_lens.copy_(torch.from_numpy(lens))
    lse2 = oracle.attention(q.double().numpy(), *planes, batch.offsets, lens, batch.table, 128 ** -0.5)[1]
    ld.copy_(torch.from_numpy(lse2.astype(np.float32)))
    graph.replay()
    torch.cuda.synchronize()
    want, bound = oracle.kv_weights(q.double().numpy(), lse2.astype(np.float32).astype(np.float64), w, planes[0],
                                    planes[1], batch.offsets, lens, batch.table, 128 ** -0.5)
    assert np.all(np.abs(wd.cpu().numpy() - want) <= bound)


@pytest.mark.parametrize("window", [1 << 30, (1 << 31) - 2, (1 << 31) - 1])
@pytest.mark.parametrize("D,group,pairs", [(128, 4, [(100, 40), (0, 5), (700, 1)]), (64, 3, [(0, 300), (130, 2)]),
                                           (256, 2, [(9, 70)])])
def test_a_window_past_every_place_hides_nothing(window, D, group, pairs):
    """The largest windows, which end past the largest place, give what no window gives."""
    rng = np.random.default_rng(19)
    batch, planes, q, lse, w = setup(rng, pairs, 16, 2, group, D, "bf16")
    none = call(batch, planes, q, lse, w, 0, 0.5)[0]
    assert torch.equal(call(batch, planes, q, lse, w, window, 0.5)[0], none)
    check(np.random.default_rng(20), pairs, 16, 2, group, D, "bf16", window=window, decay=0.5)


@pytest.mark.parametrize("page", [-1, -2, -3, -(1 << 31), (1 << 31) - 1])
@pytest.mark.parametrize("pairs", [[(100, 1), (40, 1)], [(300, 20), (40, 3)], [(2, 300), (40, 1)]])
def test_every_page_out_of_range_is_reported(page, pairs):
    rng = np.random.default_rng(21)

    def edit(b):
        b.table[0, 2] = page
    check(rng, pairs, 16, 2, 2, 128, "bf16", edit=edit, err=moe.DEVERR_PAGE)
    check(rng, pairs, 64, 1, 3, 64, "f16", edit=lambda b: b.table.__setitem__((0, 0), page), err=moe.DEVERR_PAGE)


@pytest.mark.parametrize("length", [-1, -(1 << 31), 3 - (1 << 31)])
@pytest.mark.parametrize("window", [0, 20])
def test_lengths_below_the_new_tokens(length, window):
    rng = np.random.default_rng(22)

    def edit(b):
        b.lens[1] = length
    check(rng, [(100, 6), (30, 6), (7, 2)], 16, 2, 3, 64, "bf16", window=window, edit=edit, err=moe.DEVERR_PAGE)
