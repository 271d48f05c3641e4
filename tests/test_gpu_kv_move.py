"""moe_kv_keep_e4m3 and moe_kv_evict_e4m3 against the oracle, bit for bit."""
import numpy as np
import pytest
import torch

import nvfp4_grouped_gemm_gb300 as moe
from oracle import serving as oracle
from serving_util import Batch, cache_planes, device_cache, zeros_ws

pytestmark = pytest.mark.gpu


def same_codes(got, want):
    """Equal codes; any NaN code equals any other."""
    got, want = got.cpu().numpy(), want
    nan = ((got & 0x7F) == 0x7F) & ((want & 0x7F) == 0x7F)
    assert np.array_equal(got[~nan], want[~nan])


def same_planes(cache, planes):
    same_codes(cache.k_codes, planes[0])
    assert np.array_equal(cache.k_scales.cpu().numpy(), planes[1])
    same_codes(cache.v_codes, planes[2])
    assert np.array_equal(cache.v_scales.cpu().numpy(), planes[3])


def loud(rng, planes):
    """Scales of a page and head anything in a wide range, not only powers of two."""
    return (planes[0], (2.0 ** rng.uniform(-9, 2, planes[1].shape)).astype(np.float32), planes[2],
            (2.0 ** rng.integers(-12, 9, planes[3].shape)).astype(np.float32))


# ---- keep ---------------------------------------------------------------------------------
def keep(rng, pairs, lists, page, heads, D, n_keep=None, edit=None, err=0, width=None):
    batch = Batch(rng, pairs, page)
    if edit:
        edit(batch)
    planes = loud(rng, cache_planes(rng, batch.num_pages, heads, page, D))
    width = max(map(len, lists)) if width is None else width
    table = np.full((len(pairs), width), -1, np.int32)
    for b, v in enumerate(lists):
        table[b, :len(v)] = v
    counts = np.array([len(v) for v in lists] if n_keep is None else n_keep, np.int32)
    cache = device_cache(planes)
    new_lens, ws = torch.full((len(pairs),), -9, dtype=torch.int32, device="cuda"), zeros_ws(moe.kv_keep_workspace_bytes())
    moe.moe_kv_keep_e4m3(cache, batch.device(), torch.from_numpy(table).cuda(), torch.from_numpy(counts).cuda(),
                         new_lens, ws)
    for c, s in ((planes[0], planes[1]), (planes[2], planes[3])):
        lens, cut = oracle.kv_keep(c, s, table, counts, batch.offsets, batch.lens, batch.table)
    assert moe.get_device_error(ws) == err
    same_planes(cache, planes)
    assert np.array_equal(new_lens.cpu().numpy(), lens)
    return lens


def paths(rng, pairs):
    return [sorted(rng.choice(n, rng.integers(0, n + 1), replace=False).tolist()) if n else [] for _, n in pairs]


@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("D,heads", [(64, 3), (128, 2), (256, 1)])
def test_paths_of_ragged_trees(page, D, heads):
    rng = np.random.default_rng(page + D)
    pairs = [(0, 1), (0, 9), (page - 1, 1), (page - 1, 40), (100, 0), (5, 2 * page + 3), (333, 17), (page, page), (0, 0)]
    for _ in range(2):
        keep(rng, pairs, paths(rng, pairs), page, heads, D)


def test_lists_that_keep_all_none_or_the_last():
    rng = np.random.default_rng(2)
    pairs = [(30, 6), (30, 6), (30, 6), (30, 6), (7, 70)]
    lens = keep(rng, pairs, [list(range(6)), [], [5], [0], [69]], 16, 2, 128)
    assert lens.tolist() == [36, 30, 31, 31, 8]


def test_long_lists():
    rng = np.random.default_rng(3)
    pairs = [(17, 900), (0, 700)]
    keep(rng, pairs, paths(rng, pairs), 32, 2, 64)


def test_lists_end_where_they_do_not_ascend():
    rng = np.random.default_rng(4)
    pairs = [(20, 8)] * 6
    lists = [[0, 3, 3, 5], [2, 1], [0, 8], [-1, 2], [4, 6, 7], [1, 2, 3]]
    lens = keep(rng, pairs, lists, 16, 2, 64, err=moe.DEVERR_TOKEN)
    assert lens.tolist() == [22, 21, 21, 20, 23, 23]


def test_counts_outside_the_list():
    rng = np.random.default_rng(5)
    keep(rng, [(20, 8), (20, 8), (3, 4)], [[1, 5], [0, 2], [3, 0]], 16, 1, 64, n_keep=[-3, 2, 1])
    keep(rng, [(20, 8), (20, 8)], [[1, 5], [0, 2]], 16, 1, 64, n_keep=[9, 2])
    keep(rng, [(20, 8)], [[]], 16, 1, 64, width=0)


def test_pages_out_of_range_and_bad_lengths():
    rng = np.random.default_rng(6)

    def edit(b):
        b.table[0, 2] = -1                    # a source page
        b.table[1, 1] = b.num_pages           # a target page
        b.lens[2] = 3                         # more new tokens than tokens
        b.lens[3] = 400                       # longer than the table
    keep(rng, [(16, 40), (16, 40), (0, 9), (30, 4), (30, 4)],
         [[0, 2, 17, 20, 39], [1, 2, 5, 20], [1, 2], [1, 3], [2, 3]], 16, 2, 64, edit=edit, err=moe.DEVERR_PAGE)


def test_kept_codes_are_bits_where_the_scale_stays():
    """NaN codes, and codes whose page's scale does not change, move as they are."""
    rng = np.random.default_rng(7)
    batch = Batch(rng, [(3, 10)], 16)
    planes = cache_planes(rng, batch.num_pages, 1, 16, 64)
    planes[0][:] = rng.integers(0, 256, planes[0].shape)
    cache = device_cache(planes)
    lens = torch.empty(1, dtype=torch.int32, device="cuda")
    ws = zeros_ws(moe.kv_keep_workspace_bytes())
    moe.moe_kv_keep_e4m3(cache, batch.device(), torch.tensor([[2, 4, 9]], dtype=torch.int32).cuda(),
                         torch.tensor([3], dtype=torch.int32).cuda(), lens, ws)
    page = batch.table[0, 0]
    assert np.array_equal(cache.k_codes[page, 0, 3:6].cpu().numpy(), planes[0][page, 0, [5, 7, 12]])


# ---- evict --------------------------------------------------------------------------------
def weights_of(rng, shape):
    w = np.exp(3 * rng.standard_normal(shape)).astype(np.float32)
    w[rng.random(shape) < 0.3] = 0                               # ties
    return w


def evict(rng, lens, budgets, page, heads, D, width=None, first=0, recent=0, edit=None, edit_w=None, err=0,
          none=False, dst_edit=None):
    width = max(budgets) if width is None else width
    cols = -(-width // page)
    batch = Batch(rng, [(n, 0) for n in lens], page, spare=2 + cols * len(lens))
    free = [p for p in range(batch.num_pages) if p not in
            {int(v) for b, n in enumerate(lens) for v in batch.table[b, :-(-n // page)]}]
    dst = np.array(free[:cols * len(lens)], np.int32).reshape(len(lens), cols)
    if edit:
        edit(batch)
    if dst_edit:
        dst_edit(dst)
    planes = loud(rng, cache_planes(rng, batch.num_pages, heads, page, D))
    w = weights_of(rng, (batch.num_pages, heads, page))
    if edit_w:
        edit_w(w, batch)
    cache, weights = device_cache(planes), torch.from_numpy(w).cuda()
    kept = torch.full((len(lens), heads, width), -9, dtype=torch.int32, device="cuda")
    new_lens = torch.full((len(lens),), -9, dtype=torch.int32, device="cuda")
    ws = zeros_ws(moe.kv_evict_workspace_bytes(len(lens), heads))
    b_t = None if none else torch.tensor(budgets, dtype=torch.int32, device="cuda")
    moe.moe_kv_evict_e4m3(cache, batch.device(), weights, torch.from_numpy(dst).cuda(), kept, new_lens, ws,
                          budgets=b_t, first=first, recent=recent)
    want_kept = np.full(tuple(kept.shape), -1, np.int32)
    want_lens = []
    old_w = w.copy()
    for b, n in enumerate(batch.lens):
        n, budget = int(n), width if none else budgets[b]
        if budget < 0:
            want_lens.append(n)
            continue
        n = min(max(n, 0), batch.table.shape[1] * page)
        chosen = oracle.evict_choice(old_w, n, min(budget, width), batch.table[b], first, recent)
        want_lens.append(len(chosen[0]))
        want_kept[b, :, :len(chosen[0])] = chosen
        oracle.kv_evict_copy(planes[0], planes[1], w, chosen, batch.table[b], dst[b])
        oracle.kv_evict_copy(planes[2], planes[3], None, chosen, batch.table[b], dst[b])
    assert moe.get_device_error(ws) == err
    assert np.array_equal(kept.cpu().numpy(), want_kept)
    assert np.array_equal(new_lens.cpu().numpy(), want_lens)
    assert np.array_equal(weights.cpu().numpy(), w, equal_nan=True)
    same_planes(cache, planes)
    return want_kept


@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("D,heads", [(64, 3), (128, 2), (256, 1)])
def test_budgets_of_ragged_lengths(page, D, heads):
    rng = np.random.default_rng(page + D)
    lens = [1, page - 1, page, page + 1, 3 * page + 7, 500, 0, 1500]
    evict(rng, lens, [5, page, page, 9, 2 * page, 333, 7, 1499], page, heads, D, first=2, recent=5)


def test_protected_ranges():
    rng = np.random.default_rng(21)
    for first, recent in ((0, 0), (4, 0), (0, 64), (4, 200), (300, 3), (1 << 30, 1 << 30), (100, 28)):
        evict(rng, [700, 128, 129], [128, 128, 128], 32, 2, 64, first=first, recent=recent)


def test_nothing_to_evict_and_nothing_kept():
    rng = np.random.default_rng(22)
    evict(rng, [40, 64, 10], [64, 64, 64], 16, 2, 64, first=1, recent=3)
    evict(rng, [40, 64, 10], [0, 1, 0], 16, 2, 64, width=20, first=1, recent=3)
    evict(rng, [40, 64, 10], [-1, 16, -5], 16, 2, 64, width=20)
    evict(rng, [40, 64, 10], [], 16, 2, 64, width=17, none=True)
    evict(rng, [90, 64], [80, 70], 16, 2, 64, width=31)          # budgets above the width


def test_ties_go_to_the_lower_place():
    rng = np.random.default_rng(23)

    def same(w, batch):
        w[:] = 0.25
    k = evict(rng, [300], [77], 16, 2, 64, recent=10, edit_w=same)
    assert k[0, 0].tolist() == list(range(67)) + list(range(290, 300))

    def two(w, batch):
        w[:] = rng.choice(np.array([0.0, -0.0, 1.0], np.float32), w.shape)
    evict(rng, [900, 50], [400, 20], 32, 2, 64, edit_w=two)


def test_weights_of_every_kind():
    rng = np.random.default_rng(24)

    def odd(w, batch):
        bits = rng.integers(0, 1 << 32, w.shape, dtype=np.uint64).astype(np.uint32)   # NaN, inf, negative, tiny
        w[:] = bits.view(np.float32)
        w[rng.random(w.shape) < 0.1] = np.nan
        w[rng.random(w.shape) < 0.02] = np.inf
        w[rng.random(w.shape) < 0.02] = -np.inf
    with np.errstate(invalid="ignore"):
        evict(rng, [1000, 333], [500, 320], 64, 2, 64, first=1, edit_w=odd)


def test_keys_that_do_not_fit_into_shared_memory():
    rng = np.random.default_rng(25)
    evict(rng, [60001], [4096], 128, 1, 64, first=4, recent=100)
    evict(rng, [100003, 9], [5000, 7], 128, 1, 64, first=4, recent=100)


@pytest.mark.parametrize("lens", [[4100], [8300, 5], [17000, 8193, 100], [33000, 40], [5000, 4000, 3000, 2000]])
def test_candidates_over_several_blocks(lens):
    """Long sequences' candidates are shared out: ties that cross the shares, and shares without any."""
    rng = np.random.default_rng(len(lens))

    def few(w, batch):
        w[:] = rng.choice(np.array([0.0, 1.0, 1.0 + 2.0 ** -23, 3.0], np.float32), w.shape, p=[0.6, 0.2, 0.1, 0.1])
    for edit_w in (None, few):
        evict(rng, lens, [max(1, n // 3) for n in lens], 64, 2, 64, first=1, recent=40, edit_w=edit_w)
    evict(rng, lens, [n - 1 for n in lens], 64, 1, 64, edit_w=few)


def test_pages_out_of_range():
    rng = np.random.default_rng(26)

    def edit(b):
        b.table[0, 1], b.table[1, 2] = -1, b.num_pages

    def dst_edit(d):
        d[1, 0] = -4
    evict(rng, [100, 100, 50], [90, 60, 30], 16, 2, 64, edit=edit, dst_edit=dst_edit, recent=4, err=moe.DEVERR_PAGE)

    def long_(b):
        b.lens[0] = 1 << 20
    evict(rng, [100, 40], [50, 20], 16, 1, 64, edit=long_, err=moe.DEVERR_PAGE)


def test_shared_old_pages():
    """Two sequences with a common prefix of pages, which stay as they are."""
    rng = np.random.default_rng(27)

    def edit(b):
        b.table[1, :3] = b.table[0, :3]
    evict(rng, [100, 90], [40, 50], 16, 2, 64, edit=edit, recent=8)


def test_repeated_calls_and_a_graph():
    rng = np.random.default_rng(28)
    lens, page, heads, D, width = [500, 260], 32, 2, 128, 200
    batch = Batch(rng, [(n, 0) for n in lens], page, spare=20)
    used = {int(v) for b, n in enumerate(lens) for v in batch.table[b, :-(-n // page)]}
    free = [p for p in range(batch.num_pages) if p not in used]
    dst = torch.tensor(np.array(free[:14], np.int32).reshape(2, 7)).cuda()
    planes = cache_planes(rng, batch.num_pages, heads, page, D)
    cache, weights = device_cache(planes), torch.from_numpy(weights_of(rng, (batch.num_pages, heads, page))).cuda()
    kept = torch.empty(2, heads, width, dtype=torch.int32, device="cuda")
    new_lens, ws, dev = torch.empty(2, dtype=torch.int32, device="cuda"), zeros_ws(moe.kv_evict_workspace_bytes(2, heads)), batch.device()
    moe.moe_kv_evict_e4m3(cache, dev, weights, dst, kept, new_lens, ws, recent=9)
    first = [t.clone() for t in (cache.k_codes, cache.v_codes, cache.k_scales, weights, kept, new_lens)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        moe.moe_kv_evict_e4m3(cache, dev, weights, dst, kept, new_lens, ws, recent=9)
    kept.zero_()
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    for t, was in zip((cache.k_codes, cache.v_codes, cache.k_scales, weights, kept, new_lens), first):
        assert torch.equal(t, was)


@pytest.mark.parametrize("page,D,heads", [(16, 64, 2), (64, 128, 1), (128, 256, 1)])
def test_pages_copied_from_scales_of_zero(page, D, heads):
    """A page of the copy has the largest of its tokens' scales, also where that is 0: what was 0 stays 0 on
    pages whose scales were others before."""
    rng = np.random.default_rng(29)
    lens, budgets = [3 * page, 2 * page + 5, 2 * page], [2 * page + 3, 2 * page, page + 1]
    batch = Batch(rng, [(n, 0) for n in lens], page, spare=12)
    used = {int(v) for b, n in enumerate(lens) for v in batch.table[b, :-(-n // page)]}
    dst = np.array([p for p in range(batch.num_pages) if p not in used][:9], np.int32).reshape(3, 3)
    planes = loud(rng, cache_planes(rng, batch.num_pages, heads, page, D))
    for c in (planes[0], planes[2]):                             # no sign to lose, no NaN
        c &= 0x77
    mine = batch.table[0, :3]
    planes[1][mine] = planes[3][mine] = 0                        # all of the first sequence
    planes[1][batch.table[1, 0]] = 0                             # a page of the second, of its keys only
    w = weights_of(rng, (batch.num_pages, heads, page))
    cache, weights = device_cache(planes), torch.from_numpy(w).cuda()
    kept = torch.empty(3, heads, 2 * page + 3, dtype=torch.int32, device="cuda")
    new_lens = torch.empty(3, dtype=torch.int32, device="cuda")
    ws = zeros_ws(moe.kv_evict_workspace_bytes(3, heads))
    moe.moe_kv_evict_e4m3(cache, batch.device(), weights, torch.from_numpy(dst).cuda(), kept, new_lens, ws,
                          budgets=torch.tensor(budgets, dtype=torch.int32, device="cuda"), first=1, recent=3)
    for b, n in enumerate(lens):
        chosen = oracle.evict_choice(w, n, budgets[b], batch.table[b], 1, 3)
        oracle.kv_evict_copy(planes[0], planes[1], None, chosen, batch.table[b], dst[b])
        oracle.kv_evict_copy(planes[2], planes[3], None, chosen, batch.table[b], dst[b])
    assert moe.get_device_error(ws) == 0
    assert np.all(planes[1][dst[0]] == 0) and np.all(planes[3][dst[0]] == 0)
    same_planes(cache, planes)


@pytest.mark.parametrize("length", [-1, -(1 << 31), 8 - (1 << 31), (1 << 31) - 1])
def test_keep_with_lengths_of_any_value(length):
    """Lengths below the number of new tokens, also where their difference leaves 32 bits, and above the table."""
    rng = np.random.default_rng(30)

    def edit(b):
        b.lens[1] = length
    lens = keep(rng, [(30, 9), (30, 9), (5, 40)], [[1, 4, 8], [0, 4, 8], [3, 39]], 16, 2, 64, edit=edit, err=moe.DEVERR_PAGE)
    assert lens.tolist() == [33, length, 7]
