"""moe_verify_draft against the oracle's Python integers: every id and count equal."""
import numpy as np
import pytest
import torch

import nvfp4_grouped_gemm_gb300 as moe
from oracle import serving as oracle
from serving_util import DT, zeros_ws

pytestmark = pytest.mark.gpu


def softmax(x):
    e = np.exp(x - x.max(-1, keepdims=True))
    return (e / e.sum(-1, keepdims=True)).astype(np.float32)


def draw(rng, B, n, V, dtype, sharp=2.0, near=0.5):
    logits = rng.standard_normal((B, n + 1, V)) * sharp
    target = torch.from_numpy(softmax(logits)).to(DT[dtype])
    draft = torch.from_numpy(softmax(logits[:, :n] + rng.standard_normal((B, n, V)) * near)).to(DT[dtype])
    ids = np.zeros((B, n), np.int32)
    for b in range(B):
        for i in range(n):
            p = draft[b, i].double().numpy()
            ids[b, i] = rng.choice(V, p=p / p.sum())
    return ids, target, draft, rng.uniform(size=(B, n)).astype(np.float32), rng.uniform(size=B).astype(np.float32)


def check(ids, target, draft, ua, us, n_draft=None, err=0, calls=2):
    B, n = ids.shape
    V = target.shape[2]
    want = oracle.verify_draft(ids, n_draft, target.float().numpy(),
                               None if draft is None else draft.float().numpy(), ua, us)
    out = torch.full((B, n + 1), 99, dtype=torch.int32, device="cuda")
    cnt = torch.full((B,), 99, dtype=torch.int32, device="cuda")
    ws = zeros_ws(moe.verify_workspace_bytes(B, V))
    c = lambda a: None if a is None else torch.from_numpy(a).cuda()   # noqa: E731
    for _ in range(calls):
        moe.moe_verify_draft(c(ids), target.cuda(), c(ua), c(us), out, cnt, ws,
                             draft_probs=None if draft is None else draft.cuda(), n_draft=c(n_draft))
    assert moe.get_device_error(ws) == err
    assert np.array_equal(cnt.cpu().numpy(), want[1])
    assert np.array_equal(out.cpu().numpy(), want[0])
    return want


@pytest.mark.parametrize("B,n,V,dtype", [(1, 4, 3203, "f32"), (5, 8, 1001, "bf16"), (3, 1, 7, "f16"),
                                         (2, 3, 20000, "f32"), (1, 2, 1, "f32"), (40, 5, 129, "f32"),
                                         (1, 1, 100003, "bf16"), (3, 2, 32768, "f16")])
def test_sizes_and_types(B, n, V, dtype):
    rng = np.random.default_rng(B + n + V)
    ids, t, d, ua, us = draw(rng, B, n, V, dtype)
    check(ids, t, d, ua, us)
    check(ids, t, None, ua, us)
    check(ids, t, d, ua, us, n_draft=rng.integers(0, n + 1, B).astype(np.int32))


def test_many_random_numbers_on_a_small_vocabulary():
    rng = np.random.default_rng(1)
    ids, t, d, ua, us = draw(rng, 600, 3, 11, "f32", near=1.5)
    counts = check(ids, t, d, ua, us)[1]
    assert len(set(counts.tolist())) == 4            # every number of accepted tokens occurs
    check(ids, t, None, ua, us)


def test_the_edges_of_the_random_numbers():
    rng = np.random.default_rng(2)
    ids, t, d, ua, us = draw(rng, 6, 2, 50, "f32")
    us[:] = [0.0, 1.0, np.float32(1 - 2.0 ** -24), -0.5, 2.0, np.nan]
    us_ref = us.copy()
    us_ref[5] = 0
    B, n = ids.shape
    for ua_value in (0.0, 1.0):
        ua[:] = ua_value
        want = oracle.verify_draft(ids, None, t.numpy(), d.numpy(), ua, us_ref)
        out = torch.empty(B, n + 1, dtype=torch.int32, device="cuda")
        cnt = torch.empty(B, dtype=torch.int32, device="cuda")
        ws = zeros_ws(moe.verify_workspace_bytes(B, 50))
        moe.moe_verify_draft(torch.from_numpy(ids).cuda(), t.cuda(), torch.from_numpy(ua).cuda(),
                             torch.from_numpy(us).cuda(), out, cnt, ws, draft_probs=d.cuda())
        assert np.array_equal(out.cpu().numpy(), want[0]) and np.array_equal(cnt.cpu().numpy(), want[1])


def test_no_drafts_zero_rows_and_equal_rows():
    rng = np.random.default_rng(3)
    ids, t, d, ua, us = draw(rng, 4, 2, 300, "f32")
    check(np.zeros((4, 0), np.int32), t[:, :1], None, ua[:, :0], us)
    # the draft equals the target and the random number still refuses: falls back to the target
    ua[:] = 1.0
    check(ids, t, t[:, :2].clone(), ua, us)
    # a target without mass: no token to draw
    t[1] = 0
    want = check(ids, t, d, ua, us, err=moe.DEVERR_PROBS)
    assert want[0][1, want[1][1]] == -1
    # NaN and negative entries count as nothing
    t = t.clone()
    t[0, :, 3], t[0, :, 4] = float("nan"), -1.0
    check(ids[:1], t[:1], d[:1], ua[:1], us[:1])


def test_a_single_heavy_token_and_the_last_index():
    V = 70001
    t = torch.zeros(2, 2, V)
    t[0, :, V - 1], t[1, :, 0] = 1.0, 1.0
    ids = np.array([[5], [0]], np.int32)
    want = check(ids, t, None, np.array([[0.5], [0.5]], np.float32), np.array([0.999, 0.0], np.float32))
    assert want[0].tolist() == [[V - 1, -1], [0, 0]]


def test_ids_outside_the_vocabulary_are_refused():
    rng = np.random.default_rng(4)
    ids, t, d, ua, us = draw(rng, 3, 2, 40, "f32")
    ids[0, 0], ids[1, 1] = 40, -1
    check(ids, t, d, ua * 0, us, err=moe.DEVERR_TOKEN)
    check(ids, t, None, ua * 0, us, err=moe.DEVERR_TOKEN)


def test_padded_rows():
    """Rows of a padded vocabulary: the padding is not read."""
    rng = np.random.default_rng(5)
    ids, t, d, ua, us = draw(rng, 3, 2, 333, "f32")
    tp = torch.full((3, 3, 400), float("nan"))
    dp = torch.full((3, 2, 350), float("nan"))
    tp[..., :333], dp[..., :333] = t, d
    want = oracle.verify_draft(ids, None, t.numpy(), d.numpy(), ua, us)
    out = torch.empty(3, 3, dtype=torch.int32, device="cuda")
    cnt = torch.empty(3, dtype=torch.int32, device="cuda")
    moe.moe_verify_draft(torch.from_numpy(ids).cuda(), tp.cuda()[..., :333], torch.from_numpy(ua).cuda(),
                         torch.from_numpy(us).cuda(), out, cnt, zeros_ws(moe.verify_workspace_bytes(3, 333)),
                         draft_probs=dp.cuda()[..., :333])
    assert np.array_equal(out.cpu().numpy(), want[0]) and np.array_equal(cnt.cpu().numpy(), want[1])


@pytest.mark.parametrize("B,V,dtype", [(64, 20011, "f32"), (130, 20011, "bf16"), (61, 41000, "f16"),
                                       (130, 24576, "f32")])
def test_rows_of_several_chunks_per_block(B, V, dtype):
    """Batches large enough for the larger chunks, one and several of them per block."""
    rng = np.random.default_rng(B + V)
    ids, t, d, ua, us = draw(rng, B, 2, V, dtype)
    check(ids, t, d, ua, us, n_draft=rng.integers(0, 3, B).astype(np.int32), calls=1)
    check(ids, t, None, ua, us, calls=1)
    # nothing left after the difference: every chunk of the target is summed again
    check(ids, t, t[:, :2].clone(), np.ones_like(ua), us)


def test_nothing_left_after_the_difference_in_a_long_row():
    rng = np.random.default_rng(6)
    ids, t, _, ua, us = draw(rng, 3, 2, 9001, "f32")
    check(ids, t, t[:, :2].clone(), np.ones_like(ua), us)
