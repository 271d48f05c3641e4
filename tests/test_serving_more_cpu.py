"""The operators around trees, eviction and norms without a GPU: their oracle against facts outside
itself, and the host checks of the C ABI and of the Python binding."""
import ctypes
import math

import numpy as np
import pytest
import torch

import nvfp4_grouped_gemm_gb300 as moe
from nvfp4_grouped_gemm_gb300 import _native
from oracle import serving as oracle


# ---- the oracle ---------------------------------------------------------------------
def test_a_chain_of_bits_is_causal():
    js = np.arange(40)
    chain = oracle.tree_sees([(2 << i) - 1 for i in range(9)], 9)
    for window in (0, 1, 5, 30, 100):
        for i in range(9):
            assert np.array_equal(chain(js, 31, i, window), oracle.causal_sees(js, 31, i, window))


def test_weights_oracle_against_a_dense_softmax():
    rng = np.random.default_rng(0)
    P, D, L, n = 16, 64, 37, 4
    kc = rng.integers(0, 120, (3, 2, P, D), dtype=np.uint8)
    ks = rng.uniform(0.005, 0.02, (3, 2)).astype(np.float32)
    q = rng.standard_normal((n, 4, D))
    table = np.array([[2, 0, 1]], np.int32)
    lse = oracle.attention(q, kc, ks, kc, ks, [0, n], [L], table, 0.1)[1]
    w = rng.random((3, 2, P)).astype(np.float32)
    got, _ = oracle.kv_weights(q, lse, w, kc, ks, [0, n], [L], table, 0.1, decay=0.5)
    for h in range(2):
        K = torch.from_numpy((oracle.E4M3[kc[[2, 0, 1], h]] * ks[[2, 0, 1], h].astype(np.float64)[:, None, None]).reshape(-1, D)[:L])
        total = torch.zeros(L, dtype=torch.float64)
        for t in range(n):
            seen = L - n + t + 1
            for r in (2 * h, 2 * h + 1):
                total[:seen] += torch.softmax(K[:seen] @ torch.from_numpy(q[t, r]) * 0.1, 0)
        old = torch.from_numpy(w[[2, 0, 1], h].reshape(-1)[:L - n]).double()
        total[:L - n] += 0.5 * old
        assert np.allclose(got[[2, 0, 1], h].reshape(-1)[:L], total.numpy())


def test_choice_oracle_against_a_stable_sort():
    rng = np.random.default_rng(1)
    w = rng.choice(np.array([0.0, 1.0, 2.0], np.float32), (4, 2, 16))
    table = np.array([3, 1, 0, 2])
    kept = oracle.evict_choice(w, 60, 20, table, 2, 5)
    for h in range(2):
        flat = torch.from_numpy(w[table, h].reshape(-1)[:60].copy())
        flat[:2] = flat[55:] = 9
        assert kept[h] == sorted(torch.sort(flat, descending=True, stable=True).indices[:20].tolist())


def test_keep_oracle_moves_tokens_and_grows_scales():
    codes = np.full((2, 1, 16, 64), 0x38, np.uint8)              # 1.0
    scales = np.array([[1.0], [4.0]], np.float32)
    codes[1, 0, 3] = 0x40                                        # 2.0 * 4
    lens, cut = oracle.kv_keep(codes, scales, np.array([[0, 8]]), np.array([2]), [0, 9], [20], np.array([[0, 1]]))
    assert lens.tolist() == [13] and not cut
    assert scales[0, 0] == 4.0                                   # place 12 <- place 19, page 0 <- page 1
    assert np.all(oracle.E4M3[codes[0, 0, 12]] * 4 == 8.0) and np.all(oracle.E4M3[codes[0, 0, :12]] * 4 == 1.0)


def test_norm_oracle_against_torch():
    rng = np.random.default_rng(2)
    y, res, g, w = (torch.from_numpy(rng.standard_normal(s)) for s in ((5, 48), (5, 48), (5, 1), (48,)))
    r, n, _, _ = oracle.residual_norm(y.numpy(), res.numpy(), w.numpy(), w.numpy(), g.numpy(), True, 0.5, 1e-6, 1.0)
    norm = lambda x: torch.nn.functional.rms_norm(x, (48,), w + 1, 1e-6)      # noqa: E731
    want = res + 0.5 * torch.sigmoid(g) * norm(y)
    assert torch.allclose(torch.from_numpy(r), want) and torch.allclose(torch.from_numpy(n), norm(want))


# ---- refusals of the C ABI -----------------------------------------------------------
@pytest.fixture(scope="module")
def lib():
    import os
    if not os.path.exists(_native.lib_path()):
        import nvfp4_grouped_gemm_gb300.build as b
        b.build()
    return _native.load()


def _cache(**kw):
    c = dict(k_codes=256, v_codes=256, k_scales=256, v_scales=256, num_pages=4, kv_heads=2,
             page_size=16, head_dim=128, page_stride=2 * 16 * 128)
    c.update(kw)
    return _native.KvCache(*[c[n] for n, _ in _native.KvCache._fields_])


def _batch(**kw):
    b = dict(q_offsets=256, seq_lens=256, page_table=256, B=2, max_pages=3, table_stride=3)
    b.update(kw)
    return _native.SeqBatch(*[b[n] for n, _ in _native.SeqBatch._fields_])


def _with(kw, *parts):
    for k, v in kw.items():
        next(p for p in parts if k in p)[k] = v
    return parts


def _tree(lib, cache=None, batch=None, **kw):
    a, b = _with(kw, dict(q=256, qs=1024, T=4, qh=8, dt=0),
                 dict(mask=256, words=2, ms=2, scale=0.1, window=0, out=256, os=1024, lse=None, ws=256, nb=1 << 40, s=None))
    return lib.moe_attention_tree_e4m3(*a.values(), ctypes.byref(cache or _cache()), ctypes.byref(batch or _batch()),
                                       *b.values())


def _keep(lib, cache=None, batch=None, **kw):
    (a,) = _with(kw, dict(keep=256, n=256, width=3, lens=512, ws=256, nb=1 << 40, s=None))
    return lib.moe_kv_keep_e4m3(ctypes.byref(cache or _cache()), ctypes.byref(batch or _batch()), *a.values())


def _weights(lib, cache=None, batch=None, **kw):
    a, b = _with(kw, dict(q=256, qs=1024, T=4, qh=8, dt=0, lse=256),
                 dict(scale=0.1, window=0, decay=1.0, w=256, out=256, ws=256, nb=1 << 40, s=None))
    return lib.moe_kv_weights_e4m3(*a.values(), ctypes.byref(cache or _cache()), ctypes.byref(batch or _batch()),
                                   *b.values())


def _evict(lib, cache=None, batch=None, **kw):
    (a,) = _with(kw, dict(w=256, dst=2048, ds=2, budgets=None, width=32, first=0, recent=0, kept=256, lens=512, ws=256,
                          nb=1 << 40, s=None))
    return lib.moe_kv_evict_e4m3(ctypes.byref(cache or _cache()), ctypes.byref(batch or _batch()), *a.values())


CALLS = [_tree, _keep, _weights, _evict]


@pytest.mark.parametrize("call", CALLS)
@pytest.mark.parametrize("kw,status", [
    (dict(k_codes=None), 1), (dict(v_scales=None), 1), (dict(k_codes=264), 1), (dict(num_pages=0), 1),
    (dict(kv_heads=-1), 1), (dict(page_size=48), 2), (dict(page_size=256, page_stride=1 << 20), 2), (dict(head_dim=96), 2),
    (dict(page_stride=4095), 1), (dict(page_stride=4096 + 8), 1)])
def test_a_bad_cache_is_refused(lib, call, kw, status):
    assert call(lib, cache=_cache(**kw)) == status


@pytest.mark.parametrize("call", CALLS)
@pytest.mark.parametrize("kw,status", [
    (dict(q_offsets=None), 1), (dict(seq_lens=None), 1), (dict(page_table=None), 1), (dict(B=0), 1),
    (dict(max_pages=0), 1), (dict(table_stride=2), 1), (dict(B=70000), 2),
    (dict(max_pages=1 << 24, table_stride=1 << 24), 0)])
def test_a_bad_batch_is_refused(lib, call, kw, status):
    if status == 0:                  # 2^24 pages of 128 tokens are more than 2^30 places
        assert call(lib, batch=_batch(**kw), cache=_cache(page_size=128, page_stride=2 * 128 * 128)) == 2
    else:
        assert call(lib, batch=_batch(**kw)) == status


@pytest.mark.parametrize("kw,status", [
    (dict(T=0), 1), (dict(dt=2), 1), (dict(q=None), 1), (dict(q=264), 1), (dict(qh=7), 1), (dict(scale=0.0), 1),
    (dict(scale=math.nan), 1), (dict(window=-1), 1), (dict(out=None), 1), (dict(os=1023), 1), (dict(lse=258), 1),
    (dict(mask=None), 1), (dict(mask=258), 1), (dict(words=0), 1), (dict(words=-1), 1), (dict(ms=1), 1),
    (dict(words=9, ms=9), 2), (dict(ws=None), 3), (dict(ws=128), 3), (dict(nb=0), 3)])
def test_tree_refusals(lib, kw, status):
    assert _tree(lib, **kw) == status


@pytest.mark.parametrize("kw,status", [
    (dict(keep=None), 1), (dict(keep=258), 1), (dict(n=None), 1), (dict(n=255), 1), (dict(width=-1), 1), (dict(width=(1 << 30) + 1), 2),
    (dict(lens=None), 1), (dict(lens=256), 1), (dict(n=512), 1), (dict(keep=512), 1), (dict(ws=None), 3), (dict(nb=255), 3)])
def test_keep_refusals(lib, kw, status):
    assert _keep(lib, **kw) == status


@pytest.mark.parametrize("kw,status", [
    (dict(T=0), 1), (dict(dt=2), 1), (dict(q=None), 1), (dict(q=264), 1), (dict(qs=1020), 1), (dict(qh=7), 1),
    (dict(lse=None), 1), (dict(lse=258), 1), (dict(scale=-1.0), 1), (dict(scale=math.inf), 1), (dict(window=-1), 1),
    (dict(decay=-0.1), 1), (dict(decay=1.5), 1), (dict(decay=math.nan), 1), (dict(w=None), 1), (dict(out=None), 1),
    (dict(w=264), 1), (dict(out=260), 1), (dict(T=1 << 24), 2), (dict(ws=None), 3), (dict(nb=0), 3)])
def test_weights_refusals(lib, kw, status):
    assert _weights(lib, **kw) == status


@pytest.mark.parametrize("kw,status", [
    (dict(w=None), 1), (dict(w=258), 1), (dict(dst=None), 1), (dict(ds=1), 1), (dict(width=0), 1), (dict(width=-3), 1),
    (dict(width=33), 1), (dict(first=-1), 1), (dict(recent=-1), 1), (dict(kept=None), 1), (dict(kept=257), 1),
    (dict(budgets=258), 1), (dict(lens=None), 1), (dict(lens=256), 1), (dict(budgets=512), 1), (dict(kept=512), 1), (dict(dst=1024), 1),
    (dict(width=(1 << 30) + 1, ds=1 << 28), 2),
    (dict(width=1 << 30, ds=1 << 26, ), 0), (dict(ws=None), 3), (dict(nb=0), 3)])
def test_evict_refusals(lib, kw, status):
    if status == 0:                  # more pages of copies than a grid has blocks
        assert _evict(lib, batch=_batch(B=60000), **kw) == 2
    else:
        assert _evict(lib, batch=_batch(page_table=1024), **kw) == status


@pytest.mark.parametrize("kw,status", [
    (dict(T=0), 1), (dict(T=(1 << 30) + 1), 2), (dict(H=0), 1), (dict(H=32769, ys=1 << 20, rs=1 << 20, os=1 << 20, ns=1 << 20), 2), (dict(r=None), 1),
    (dict(r=257), 1), (dict(y=257), 1), (dict(y=258, yd=2), 1), (dict(out=None, n=None), 1), (dict(out=None, n=None, pre=None), 1),
    (dict(yd=3), 1), (dict(rd=-1), 1), (dict(nd=5), 1), (dict(wd=7), 1), (dict(gd=4), 1), (dict(ys=63), 1), (dict(rs=63), 1),
    (dict(os=63), 1), (dict(ns=0), 1), (dict(y=None), 1), (dict(y=None, post=None), 1), (dict(n=None), 1),
    (dict(post=257), 1), (dict(pre=258, wd=2), 1), (dict(g=257), 1), (dict(gi=2), 1), (dict(gs=-1), 1),
    (dict(eps=-1.0), 1), (dict(eps=math.nan), 1), (dict(eps=math.inf), 1), (dict(scale=math.nan), 1), (dict(off=math.inf), 1),
    # outputs upon inputs of another stride or type, or upon one another
    (dict(out=1024, os=72), 1), (dict(out=512), 1), (dict(n=512, nd=1), 1), (dict(n=1024, ns=128), 1), (dict(n=2048), 1),
    (dict(g=2048), 1), (dict(g=4096), 1), (dict(pre=4096), 1), (dict(post=2048), 1)])
def test_norm_refusals(lib, kw, status):
    a = dict(y=512, ys=64, yd=2, r=1024, rs=64, out=2048, os=64, rd=0, n=4096, ns=64, nd=0, T=2, H=64, post=256, pre=256,
             wd=0, g=256, gs=64, gi=1, gd=2, sig=0, scale=1.0, eps=1e-6, off=0.0, s=None)
    a.update(kw)
    assert lib.moe_residual_norm(*a.values()) == status


def test_workspace_sizes(lib):
    assert moe.kv_keep_workspace_bytes() >= 4
    assert moe.kv_weights_workspace_bytes(1, 32, 8, 128) >= 4
    assert moe.kv_weights_workspace_bytes(0, 32, 8, 128) == 0
    assert moe.kv_weights_workspace_bytes(4, 30, 8, 128) == 0
    assert moe.kv_weights_workspace_bytes(4, 32, 8, 96) == 0
    assert moe.kv_weights_workspace_bytes(1 << 23, 1024, 8, 128) == 0
    assert moe.kv_evict_workspace_bytes(3, 8) >= 4
    assert moe.kv_evict_workspace_bytes(0, 8) == 0


def test_the_binding_refuses_host_tensors(lib, monkeypatch):
    from nvfp4_grouped_gemm_gb300 import serving
    monkeypatch.setattr(serving, "_device", lambda: 0)
    x = torch.zeros(2, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        moe.moe_residual_norm(x, x, x)
    with pytest.raises(ValueError):
        moe.moe_residual_norm(None, torch.zeros(64), torch.zeros(64))


# Addresses that lie apart by far (nothing is launched: there is no device, or the call is refused).
_FAR = [0x10000000 * i for i in range(1, 12)]


def _far_batch(**kw):
    b = dict(q_offsets=_FAR[0], seq_lens=_FAR[1], page_table=_FAR[2])
    b.update(kw)
    return _batch(**b)


@pytest.mark.parametrize("shift", [0, 4])
@pytest.mark.parametrize("on", ["seq_lens", "q_offsets", "page_table", "n", "keep"])
def test_keep_refuses_new_lengths_upon_what_it_reads(lib, on, shift):
    """Also where only a part of them lies there."""
    at = {"seq_lens": _FAR[1], "q_offsets": _FAR[0], "page_table": _FAR[2], "n": _FAR[3], "keep": _FAR[4]}
    kw = dict(n=_FAR[3], keep=_FAR[4], ws=_FAR[5])
    for lens in (at[on] + shift, at[on] - 4):
        assert _keep(lib, batch=_far_batch(), lens=lens, **kw) == 1


@pytest.mark.parametrize("on", ["seq_lens", "budgets", "page_table", "dst", "other", "w"])
@pytest.mark.parametrize("out", ["kept", "lens", "w"])
def test_evict_refuses_outputs_upon_what_it_reads_or_writes(lib, out, on):
    a = dict(w=_FAR[3], dst=_FAR[4], budgets=_FAR[5], kept=_FAR[6], lens=_FAR[7], ws=_FAR[8])
    at = dict(seq_lens=_FAR[1], page_table=_FAR[2], budgets=a["budgets"], dst=a["dst"], w=a["w"],
              other=a["lens" if out == "kept" else "kept"])[on]
    if out == on:
        return
    for shift in (0, 4, -4):
        assert _evict(lib, batch=_far_batch(), **{**a, out: at + shift}) == 1
    assert _evict(lib, batch=_far_batch(), **{**a, "nb": 0}) == 3          # (the others are no reason to refuse)


@pytest.mark.parametrize("kw", [dict(out=_FAR[3] + 64), dict(out=_FAR[3] - 16), dict(out=_FAR[4]), dict(out=_FAR[5]),
                                dict(out=_FAR[5] + 4 * 1024 * 2 - 16)])
def test_weights_refuses_new_weights_upon_a_part_of_what_it_reads(lib, kw):
    a = dict(w=_FAR[3], out=_FAR[6], lse=_FAR[4], q=_FAR[5], ws=_FAR[8])
    assert _weights(lib, batch=_far_batch(), **{**a, **kw}) == 1
    assert _weights(lib, batch=_far_batch(), **{**a, **kw, "nb": 0}) == 3


def test_the_first_and_last_bytes_of_neighbours_may_touch(lib):
    """Arrays one behind the other are not refused: without a device such a call gets as far as the launch."""
    if torch.cuda.is_available():
        pytest.skip("would launch")
    one = dict(n=_FAR[3], keep=_FAR[4], ws=_FAR[5], lens=_FAR[1] + 8)      # B = 2: right behind seq_lens
    assert _keep(lib, batch=_far_batch(), **one) == 4
    a = dict(w=_FAR[3], out=_FAR[3] + 4 * 4 * 2 * 16, lse=_FAR[4], q=_FAR[5], ws=_FAR[8])
    assert _weights(lib, batch=_far_batch(), **a) == 4
    b = dict(w=_FAR[3], dst=_FAR[4], budgets=_FAR[1] + 8, kept=_FAR[6], lens=_FAR[1] + 16, ws=_FAR[8])
    assert _evict(lib, batch=_far_batch(), **b) == 4
