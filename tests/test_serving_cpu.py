"""The serving operators without a GPU: their oracle against facts outside itself, and the
host checks of the C ABI and of the Python binding."""
import ctypes
import math

import numpy as np
import pytest
import torch

import nvfp4_grouped_gemm_gb300 as moe
from nvfp4_grouped_gemm_gb300 import _native
from oracle import serving as oracle


# ---- the oracle ---------------------------------------------------------------------
def test_e4m3_table_and_rounding_against_torch():
    codes = torch.arange(256, dtype=torch.uint8)
    want = codes.view(torch.float8_e4m3fn).float().numpy()
    assert np.array_equal(oracle.E4M3.astype(np.float32), want, equal_nan=True)
    rng = np.random.default_rng(0)
    v = np.concatenate([rng.uniform(-448, 448, 20000), 2.0 ** rng.uniform(-14, 8.8, 20000),
                        (oracle.E4M3[:126] + oracle.E4M3[1:127]) / 2, [0.0, 448.0]]).astype(np.float32)
    want = torch.from_numpy(v).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(oracle.e4m3_encode(v), want)


@pytest.mark.parametrize("a,e", [(0.0, -64), (448.0, 0), (449.0, 1), (224.0, -1), (1e-30, -64),
                                 (3e38, 119), (math.nextafter(224, 300), 0)])
def test_scale_exponent(a, e):
    assert oracle.scale_exponent(a) == e


def test_rotation_is_a_rotation_and_both_orders_agree():
    rng = np.random.default_rng(1)
    x = rng.standard_normal((5, 64)).astype(np.float32)
    ang = rng.uniform(0, 6, (5, 16))
    c, s = np.cos(ang).astype(np.float32), np.sin(ang).astype(np.float32)
    y = oracle.rotate(x, c, s, False)
    z = (x[:, :16] + 1j * x[:, 16:32]) * np.exp(1j * ang)
    assert np.allclose(y[:, :16] + 1j * y[:, 16:32], z, atol=1e-5)
    assert np.array_equal(y[:, 32:], x[:, 32:])
    inter = np.arange(32).reshape(2, 16).T.reshape(-1)           # (i, i + 16) side by side
    w = x.copy()
    w[:, :32] = x[:, inter]
    assert np.array_equal(oracle.rotate(w, c, s, True)[:, :32], y[:, inter])


def test_attention_oracle_against_a_dense_softmax():
    rng = np.random.default_rng(2)
    P, D, L, n = 16, 64, 37, 3
    kc = rng.integers(0, 120, (3, 1, P, D), dtype=np.uint8)
    vc = rng.integers(0, 120, (3, 1, P, D), dtype=np.uint8)
    ks = np.array([[0.01], [0.02], [0.005]], np.float32)
    q = rng.standard_normal((n, 2, D))
    table = np.array([[2, 0, 1]], np.int32)
    out, lse, _, _ = oracle.attention(q, kc, ks, vc, ks, [0, n], [L], table, 0.1)
    K = torch.from_numpy((oracle.E4M3[kc[[2, 0, 1], 0]] * ks[[2, 0, 1]][:, None].astype(np.float64)).reshape(-1, D)[:L])
    V = torch.from_numpy((oracle.E4M3[vc[[2, 0, 1], 0]] * ks[[2, 0, 1]][:, None].astype(np.float64)).reshape(-1, D)[:L])
    for t in range(n):
        seen = L - n + t + 1
        sc = torch.from_numpy(q[t]) @ K[:seen].T * 0.1
        assert torch.allclose(torch.softmax(sc, 1) @ V[:seen], torch.from_numpy(out[t]))
        assert torch.allclose(torch.logsumexp(sc, 1), torch.from_numpy(lse[t]))


def test_verify_oracle_follows_the_target_distribution():
    """Whatever the draft, the first token's distribution is the target's (here by exhausting a
    grid of random numbers on a small vocabulary)."""
    p = np.array([0.5, 0.25, 0.125, 0.125], np.float32)
    q = np.array([0.125, 0.5, 0.25, 0.125], np.float32)
    G = 64
    got = np.zeros(4)
    for x in range(4):
        for i in range(G):
            for j in range(G):
                ids, c = oracle.verify_draft(
                    np.array([[x]], np.int32), None, np.stack([p, p])[None], q[None, None],
                    np.array([[(i + 0.5) / G]], np.float32), np.array([(j + 0.5) / G], np.float32))
                got[ids[0, 0]] += q[x] / G / G
    assert np.allclose(got, p, atol=1.0 / G)


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


def _append(lib, cache=None, batch=None, **kw):
    a = dict(T=4, k=256, ks=256, v=256, vs=256, q=256, qs=1024, qo=256, qos=1024, qh=8, dt=0, cos=256,
             sin=256, max_pos=100, rot=128, inter=0, pos=None, ws=256, nb=256, s=None)
    a.update(kw)
    return lib.moe_kv_append_rope_e4m3(ctypes.byref(cache or _cache()), ctypes.byref(batch or _batch()),
                                       *a.values())


def _attend(lib, cache=None, batch=None, **kw):
    a = dict(q=256, qs=1024, T=4, qh=8, dt=0)
    b = dict(scale=0.1, window=0, out=256, os=1024, lse=None, ws=256, nb=1 << 40, s=None)
    for k, v in kw.items():
        (a if k in a else b)[k] = v
    return lib.moe_attention_paged_e4m3(*a.values(), ctypes.byref(cache or _cache()),
                                        ctypes.byref(batch or _batch()), *b.values())


BAD_CACHE = [(dict(k_codes=None), 1), (dict(v_scales=None), 1), (dict(k_codes=264), 1),
             (dict(num_pages=0), 1), (dict(kv_heads=-1), 1), (dict(page_size=48), 2),
             (dict(page_size=256, page_stride=1 << 20), 2), (dict(head_dim=96), 2),
             (dict(page_stride=4095), 1), (dict(page_stride=4096 + 8), 1)]
BAD_BATCH = [(dict(q_offsets=None), 1), (dict(seq_lens=None), 1), (dict(page_table=None), 1),
             (dict(B=0), 1), (dict(max_pages=0), 1), (dict(table_stride=2), 1), (dict(B=70000), 2)]


@pytest.mark.parametrize("kw,status", BAD_CACHE)
def test_a_bad_cache_is_refused(lib, kw, status):
    assert _append(lib, cache=_cache(**kw)) == status
    assert _attend(lib, cache=_cache(**kw)) == status


@pytest.mark.parametrize("kw,status", BAD_BATCH)
def test_a_bad_batch_is_refused(lib, kw, status):
    assert _append(lib, batch=_batch(**kw)) == status
    assert _attend(lib, batch=_batch(**kw)) == status


@pytest.mark.parametrize("kw,status", [
    (dict(T=0), 1), (dict(dt=2), 1), (dict(dt=7), 1), (dict(k=None), 1), (dict(k=264), 1),
    (dict(ks=255), 1), (dict(ks=260), 1), (dict(v=None), 1), (dict(vs=128), 1), (dict(qo=None), 1),
    (dict(qh=0), 1), (dict(qs=1000), 1), (dict(rot=136), 1), (dict(rot=24), 1), (dict(rot=-16), 1),
    (dict(cos=None), 1), (dict(sin=260), 1), (dict(max_pos=0), 1), (dict(ws=None), 3),
    (dict(ws=264), 3), (dict(nb=255), 3), (dict(T=1 << 24), 2)])
def test_append_refusals(lib, kw, status):
    assert _append(lib, **kw) == status


@pytest.mark.parametrize("kw,status", [
    (dict(T=0), 1), (dict(dt=2), 1), (dict(q=None), 1), (dict(q=264), 1), (dict(qh=7), 1),
    (dict(qh=0), 1), (dict(scale=0.0), 1), (dict(scale=-1.0), 1), (dict(scale=math.nan), 1),
    (dict(scale=math.inf), 1), (dict(window=-1), 1), (dict(out=None), 1), (dict(os=1023), 1),
    (dict(lse=258), 1), (dict(ws=None), 3), (dict(ws=128), 3), (dict(nb=0), 3)])
def test_attention_refusals(lib, kw, status):
    assert _attend(lib, **kw) == status


@pytest.mark.parametrize("kw,status", [
    (dict(x=None), 1), (dict(x=8), 1), (dict(xs=120), 1), (dict(xs=132), 1), (dict(xd=2), 1),
    (dict(T=0), 1), (dict(y=None), 1), (dict(y=258), 1), (dict(ys=63), 1), (dict(yd=3), 1),
    (dict(ws=None), 3), (dict(nb=0), 3)])
def test_linear_refusals(lib, kw, status):
    a = dict(x=256, xs=128, xd=0, T=2)
    b = dict(y=256, ys=64, yd=2, ws=256, nb=1 << 40, s=None)
    for k, v in kw.items():
        (a if k in a else b)[k] = v
    bank = _native.Bank(256, 256, 1, 64, 128)
    assert lib.moe_linear_nvfp4(*a.values(), ctypes.byref(bank), *b.values()) == status


@pytest.mark.parametrize("bank,status", [((None, 256, 1, 64, 128), 1), ((256, 8, 1, 64, 128), 1),
                                         ((256, 256, 2, 64, 128), 1), ((256, 256, 1, 0, 128), 1),
                                         ((256, 256, 1, 64, 112), 2), ((256, 256, 1, 64, 65568), 2)])
def test_linear_refuses_a_bad_bank(lib, bank, status):
    assert lib.moe_linear_nvfp4(256, 1 << 20, 0, 2, ctypes.byref(_native.Bank(*bank)), 256, 64, 2, 256,
                                1 << 40, None) == status


@pytest.mark.parametrize("kw,status", [
    (dict(ids=None), 1), (dict(B=0), 1), (dict(n=-1), 1), (dict(V=0), 1), (dict(t=None), 1),
    (dict(ts=99), 1), (dict(ds=99), 1), (dict(dt=3), 1), (dict(t=258), 1), (dict(ua=None), 1),
    (dict(us=None), 1), (dict(out=None), 1), (dict(cnt=None), 1), (dict(n=65), 2),
    (dict(V=(1 << 22) + 1, ts=1 << 23, ds=1 << 23), 2), (dict(B=65536), 2), (dict(ws=None), 3),
    (dict(nb=0), 3)])
def test_verify_refusals(lib, kw, status):
    a = dict(ids=256, nd=None, B=2, n=3, V=100, t=256, ts=100, d=256, ds=100, dt=2, ua=256, us=256,
             out=256, cnt=256, ws=256, nb=1 << 40, s=None)
    a.update(kw)
    assert lib.moe_verify_draft(*a.values()) == status


def test_workspace_sizes(lib):
    assert moe.kv_append_workspace_bytes() >= 4
    assert moe.attention_workspace_bytes(32, 8, 128) >= 4
    assert moe.attention_workspace_bytes(30, 8, 128) == 0
    assert moe.attention_workspace_bytes(32, 8, 96) == 0
    assert moe.linear_workspace_bytes(1, 5, 64) >= 4
    assert moe.linear_workspace_bytes(1, 5, 65) == 0
    assert moe.linear_workspace_bytes(0, 5, 64) == 0
    assert moe.verify_workspace_bytes(3, 1000) >= 4
    assert moe.verify_workspace_bytes(3, (1 << 22) + 1) == 0


def test_the_binding_refuses_host_tensors_and_wrong_shapes():
    codes = torch.zeros(4, 2, 16, 64, dtype=torch.uint8)
    scales = torch.ones(4, 2)
    with pytest.raises(ValueError):
        moe.PagedKvCache(codes, codes, scales, scales)
    with pytest.raises(TypeError):
        moe.PagedKvCache(codes.float(), codes, scales, scales)
    i = torch.zeros(3, dtype=torch.int32)
    with pytest.raises(ValueError):
        moe.SeqBatch(i, i[:2], torch.zeros(2, 4, dtype=torch.int32))
    with pytest.raises(TypeError):
        moe.SeqBatch(i, i[:2], torch.zeros(2, 4))
