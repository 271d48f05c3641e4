"""moe_attention_tree_e4m3 against the float64 oracle, within the oracle's error bound plus the
rounding of the output type."""
import numpy as np
import pytest
import torch

import nvfp4_grouped_gemm_gb300 as moe
from oracle import serving as oracle
from serving_util import Batch, activations, cache_planes, device_cache, zeros_ws

pytestmark = pytest.mark.gpu
# half a step of 8 and 11 significant bits, and half the least subnormal
ROUND = {"bf16": (2.0 ** -8, 2.0 ** -134), "f16": (2.0 ** -11, 2.0 ** -25)}


def tree_bits(rng, n):
    """Ancestors and itself of each node of a random tree, as whole numbers."""
    bits = []
    for i in range(n):
        parent = int(rng.integers(0, i)) if i and rng.random() < 0.95 else -1
        bits.append(1 << i | (bits[parent] if parent >= 0 else 0))
    return bits


def mask_of(trees, words, spare=0, junk=0):
    rows = [[(v >> 32 * w) & 0xFFFFFFFF for w in range(words)] + [junk] * spare for t in trees for v in t]
    return torch.from_numpy(np.array(rows, np.uint32).view(np.int32)).cuda()


def stale_nan(planes, batch):
    used = np.zeros((batch.num_pages, batch.page), bool)
    for b, n in enumerate(batch.lens):
        for i in range(min(int(n), batch.table.shape[1] * batch.page)):
            if 0 <= batch.table[b, i // batch.page] < batch.num_pages:
                used[batch.table[b, i // batch.page], i % batch.page] = True
    for c in (planes[0], planes[2]):
        c.transpose(0, 2, 1, 3)[~used] = 0x7F


def check(rng, pairs, page, heads, group, D, dtype, window=0, make=tree_bits, words=None, edit=None, err=0, spare=0,
          edit_planes=None, junk=0):
    batch = Batch(rng, pairs, page)
    if edit:
        edit(batch)
    planes = cache_planes(rng, batch.num_pages, heads, page, D)
    stale_nan(planes, batch)
    if edit_planes:
        edit_planes(planes, batch)
    trees = [make(rng, n) for _, n in pairs]
    words = -(-max(n for _, n in pairs) // 32) if words is None else words
    mask = mask_of(trees, words, spare, junk)[:, :words]
    seen_bits = [[v & (1 << 32 * words) - 1 for v in t] for t in trees]
    q = activations(rng, (batch.T, heads * group, D), dtype)
    want, wl, eo, el = oracle.attention(q.double().numpy(), *planes, batch.offsets, batch.lens, batch.table,
                                        D ** -0.5, window, seen_bits)
    # a table of its own width, and one so wide that many rows take the form for many rows
    for cols in (0, (1 << 20) // page):
        batch.table = np.pad(batch.table, ((0, 0), (0, cols)), constant_values=-7)
        out = torch.full((batch.T, heads * group, D), float("nan"), dtype=q.dtype, device="cuda")
        lse = torch.full((batch.T, heads * group), float("nan"), device="cuda")
        ws = zeros_ws(moe.attention_workspace_bytes(heads * group, heads, D))
        moe.moe_attention_tree_e4m3(q.cuda(), device_cache(planes), batch.device(), mask, out, ws, window=window, lse=lse)
        assert moe.get_device_error(ws) == err
        got, gl = out.double().cpu().numpy(), lse.double().cpu().numpy()
        rel, floor = ROUND[dtype]
        tol = eo + rel * (np.abs(want) + eo) + floor
        off = np.abs(got - want)
        ok = (off <= tol) | (np.isnan(got) & np.isnan(want))
        assert ok.all(), float(np.nanmax(off / tol))
        seen = wl > -np.inf
        fine = np.isfinite(wl)
        assert np.array_equal(np.isfinite(gl), fine) and np.all(gl[wl == -np.inf] == -np.inf)
        assert np.all(np.abs(gl[fine] - wl[fine]) <= el[fine] + 1e-6)
        assert np.all(got[~seen & ~np.isnan(wl)] == 0)
    return out, lse


# (rows per key head on both sides of the two forms' border, 73)
SHAPES = [(128, 64, 2, 4, "bf16", [(100, 8), (0, 3), (511, 5), (64, 16)]),
          (64, 16, 1, 5, "f16", [(0, 1), (0, 17), (33, 31), (700, 4)]),
          (256, 32, 1, 2, "bf16", [(10, 40), (200, 9)]),
          (128, 16, 1, 1, "bf16", [(5, 130)]),
          (128, 64, 1, 4, "bf16", [(0, 129), (300, 64), (3, 1), (9, 0)]),
          (64, 64, 2, 8, "f16", [(77, 100), (0, 200)]),
          (128, 128, 1, 7, "f16", [(1000, 37), (0, 150)]),
          (256, 16, 2, 7, "f16", [(1, 100), (129, 33)]),
          (64, 32, 1, 1, "bf16", [(1025, 256)]),
          (128, 32, 3, 2, "f16", [(95, 1), (0, 1), (31, 2), (63, 32), (62, 33)]),
          # more sequences than a block has threads, and segments that reach over several pieces
          (64, 16, 1, 2, "bf16", [(i % 40, 1 + i % 3) for i in range(140)]),
          (128, 64, 1, 2, "bf16", [(2500, 9), (0, 2), (1500, 4)])]


@pytest.mark.parametrize("D,page,heads,group,dtype,pairs", SHAPES)
def test_trees(D, page, heads, group, dtype, pairs):
    check(np.random.default_rng(group + D), pairs, page, heads, group, D, dtype)


@pytest.mark.parametrize("window", [1, 3, 20, 64, 130])
@pytest.mark.parametrize("D,page,heads,group,dtype,pairs", [SHAPES[0], SHAPES[2], SHAPES[4], SHAPES[5]])
def test_windows_end_at_the_row_itself(window, D, page, heads, group, dtype, pairs):
    check(np.random.default_rng(window + D), pairs, page, heads, group, D, dtype, window=window)


@pytest.mark.parametrize("D,group", [(128, 4), (64, 1), (256, 2), (128, 40)])
def test_any_bits(D, group):
    """Masks that are no trees: rows that see later tokens, not themselves, or no new token."""
    def make(rng, n):
        kinds = [0, (1 << n) - 1] if n else []
        return [int(rng.choice(2)) * 0 + (kinds[int(rng.integers(0, 2))] if rng.random() < 0.3 else
                                          int.from_bytes(rng.bytes(40), "little") & (1 << n) - 1) for _ in range(n)]
    rng = np.random.default_rng(D + group)
    for window in (0, 9):
        check(rng, [(0, 5), (40, 37), (200, 70), (0, 1), (128, 33)], 16, 2, group, D, "f16", window=window, make=make)


def test_rows_that_see_nothing():
    """No token before the new ones and an empty mask."""
    rng = np.random.default_rng(31)
    for group in (2, 30):
        out, lse = check(rng, [(0, 6), (0, 3)], 16, 1, group, 64, "bf16", make=lambda r, n: [0] * (n - 1) + [1 << n - 1])
        assert torch.all(out[0] == 0) and torch.all(torch.isinf(lse[0]))


def test_a_chain_is_the_causal_attention():
    rng = np.random.default_rng(32)
    for pairs, group, D, page in (([(300, 9), (17, 4)], 4, 128, 64), ([(300, 90), (17, 40)], 4, 64, 16)):
        batch = Batch(rng, pairs, page)
        planes = cache_planes(rng, batch.num_pages, 2, page, D)
        q = activations(rng, (batch.T, 2 * group, D), "bf16").cuda()
        cache, dev = device_cache(planes), batch.device()
        ws = zeros_ws(moe.attention_workspace_bytes(2 * group, 2, D))
        mask = mask_of([[(2 << i) - 1 for i in range(n)] for _, n in pairs], 3)
        for window in (0, 50):
            a, b = torch.empty_like(q), torch.empty_like(q)
            moe.moe_attention_paged_e4m3(q, cache, dev, a, ws, window=window)
            moe.moe_attention_tree_e4m3(q, cache, dev, mask, b, ws, window=window)
            # the same weights in f16 and f32 sums of them; where tiles are cut may differ
            assert (a.float() - b.float()).abs().max() <= 2.0 ** -7 * a.float().abs().max()


def test_bits_past_the_new_tokens_and_mask_strides():
    """Bits from n on have no meaning, rows of the mask may lie apart, and new tokens past the mask are
    seen by nobody."""
    rng = np.random.default_rng(33)

    def junk(rng_, n):
        return [v | (int.from_bytes(rng_.bytes(30), "little") << n) for v in tree_bits(rng_, n)]
    check(rng, [(20, 5), (100, 40), (64, 90)], 16, 1, 3, 64, "f16", make=junk, words=7, window=12)
    check(rng, [(20, 5), (100, 40), (64, 90)], 16, 1, 3, 128, "bf16", spare=3, junk=-1 & 0xFFFFFFFF)
    check(rng, [(20, 70), (10, 5)], 16, 1, 2, 64, "bf16", words=1)
    check(rng, [(20, 300)], 16, 1, 1, 64, "bf16", words=8)


def test_nan_codes_reach_only_the_rows_that_see_them():
    rng = np.random.default_rng(34)

    def codes(planes, batch):
        start = int(batch.lens[0]) - int(batch.offsets[1])
        for j, plane in ((start + 3, 2), (start + 5, 0), (4, 2)):
            planes[plane][batch.table[0, j // batch.page], 0, j % batch.page, 9] = 0x7F
    for n, group in ((12, 2), (40, 6)):
        for window in (0, 7):
            check(rng, [(70, n), (33, 5)], 16, 1, group, 64, "bf16", window=window, edit_planes=codes)


def test_bad_pages_and_lengths():
    rng = np.random.default_rng(35)

    def edit(b):
        b.table[0, 2], b.table[1, 0] = -1, b.num_pages
    for group in (2, 20):
        check(rng, [(100, 6), (10, 4), (40, 3)], 16, 2, group, 128, "bf16", edit=edit, err=moe.DEVERR_PAGE)


def test_a_graph_with_another_tree():
    rng = np.random.default_rng(36)
    batch = Batch(rng, [(200, 20)], 16)
    planes = cache_planes(rng, batch.num_pages, 1, 16, 128)
    q = activations(rng, (20, 4, 128), "bf16").cuda()
    cache, dev, ws = device_cache(planes), batch.device(), zeros_ws(moe.attention_workspace_bytes(4, 1, 128))
    masks = [mask_of([tree_bits(rng, 20)], 1) for _ in range(2)]
    mask, out, want = masks[0].clone(), torch.empty_like(q), torch.empty_like(q)
    moe.moe_attention_tree_e4m3(q, cache, dev, masks[1], want, ws)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        moe.moe_attention_tree_e4m3(q, cache, dev, mask, out, ws)
    mask.copy_(masks[1])
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)


@pytest.mark.parametrize("length", [-1, -(1 << 31), 3 - (1 << 31)])
@pytest.mark.parametrize("window", [0, 20])
def test_lengths_below_the_new_tokens(length, window):
    rng = np.random.default_rng(37)

    def edit(b):
        b.lens[1] = length
    for group in (2, 20):
        check(rng, [(100, 6), (30, 6), (7, 2)], 16, 2, group, 64, "bf16", window=window, edit=edit, err=moe.DEVERR_PAGE)


def used_slots(batch):
    used = np.zeros((batch.num_pages, batch.page), bool)
    for b, n in enumerate(batch.lens):
        for i in range(int(n)):
            used[batch.table[b, i // batch.page], i % batch.page] = True
    return used


@pytest.mark.parametrize("D,group,pairs", [(128, 4, [(700, 40), (90, 3)]), (64, 8, [(2500, 17), (10, 60)]), (256, 2, [(400, 30)])])
def test_repeated_calls_repeat_bit_for_bit(D, group, pairs):
    """The same bits from every call: with a used and with a new workspace, in a graph, over other stale slots."""
    rng = np.random.default_rng(38)
    batch = Batch(rng, pairs, 16)
    planes = cache_planes(rng, batch.num_pages, 2, 16, D)
    mask = mask_of([tree_bits(rng, n) for _, n in pairs], 2)
    q = activations(rng, (batch.T, 2 * group, D), "f16").cuda()
    for cols in (0, 1 << 16):                                    # few rows alone, and both forms
        batch.table = np.pad(batch.table, ((0, 0), (0, cols)), constant_values=-7)
        dev, ws = batch.device(), zeros_ws(moe.attention_workspace_bytes(2 * group, 2, D))
        want = None
        for i in range(6):
            other = [p.copy() for p in planes]
            for c in (other[0], other[2]):
                c.transpose(0, 2, 1, 3)[~used_slots(batch)] = rng.integers(0, 256)
            cache, out = device_cache(other), torch.empty_like(q)
            lse = torch.empty(q.shape[:2], device="cuda")
            space = ws if i % 2 else torch.zeros_like(ws)
            call = lambda: moe.moe_attention_tree_e4m3(q, cache, dev, mask, out, space, lse=lse)   # noqa: B023, E731
            if i < 4:
                call()
            else:
                graph = torch.cuda.CUDAGraph()
                with torch.cuda.graph(graph):
                    call()
                graph.replay()
            torch.cuda.synchronize()
            want = (out, lse) if want is None else want
            assert torch.equal(out, want[0]) and torch.equal(lse, want[1])
