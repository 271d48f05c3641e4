"""moe_residual_norm against float64, within the oracle's bound plus the rounding of the output type."""
import numpy as np
import pytest
import torch

import nvfp4_grouped_gemm_gb300 as moe
from oracle import serving as oracle
from serving_util import DT

pytestmark = pytest.mark.gpu
# half a step of the type relative to a value, and half its least subnormal
HALF = {"bf16": (2.0 ** -8, 2.0 ** -134), "f16": (2.0 ** -11, 2.0 ** -25), "f32": (2.0 ** -24, 2.0 ** -150)}


def close(got, want, err, dtype):
    rel, floor = HALF[dtype]
    tol = err + rel * (np.abs(want) + err) + floor
    bad = np.abs(got.double().cpu().numpy() - want) / tol
    assert np.all(bad <= 1), float(np.nanmax(bad))


def make(rng, T, H, y="bf16", residual="bf16", normed="bf16", post=True, pre=True, gate=None, wt="bf16", gt="f32",
         pad=0, shift=0, amp=1.0):
    """Tensors on the GPU; rows `pad` elements longer than H, starting `shift` elements in."""
    def rows(dt, a):
        x = torch.from_numpy((rng.standard_normal((T, H + pad + shift)) * a).astype(np.float32)).to(DT[dt]).cuda()
        return x[:, shift:shift + H]
    s = {"y": rows(y, 2 * amp) if y else None, "residual": rows(residual, 3 * amp)}
    s["out"] = torch.full((T, H + pad + shift), 7.0, dtype=DT[residual], device="cuda")[:, shift:shift + H]
    s["normed"] = torch.full((T, H + pad + shift), 7.0, dtype=DT[normed], device="cuda")[:, shift:shift + H] if normed else None
    for name, there in (("post_weight", post and y), ("pre_weight", pre and normed)):
        s[name] = torch.from_numpy((1 + 0.3 * rng.standard_normal(H)).astype(np.float32)).to(DT[wt]).cuda() if there else None
    shape = {None: None, "token": (T, 1), "channel": (1, H), "full": (T, H), "one": (1, 1)}[gate]
    s["gate"] = torch.from_numpy((rng.standard_normal(shape) * 2).astype(np.float32)).to(DT[gt]).cuda() if shape else None
    return s


def want(s, **kw):
    d = {k: None if v is None else v.double().cpu().numpy() for k, v in s.items()}
    return oracle.residual_norm(d["y"], d["residual"], d["post_weight"], d["pre_weight"], d["gate"],
                                kw.get("gate_sigmoid", False), kw.get("scale", 1.0), kw.get("eps", 1e-6),
                                kw.get("weight_offset", 0.0))


def names(s):
    return {v: k for k, v in DT.items()}[s.dtype]


def check(s, **kw):
    r, n, er, en = want(s, **kw)
    moe.moe_residual_norm(**s, **kw)
    if s["out"] is not None:
        close(s["out"], r, er, names(s["out"]))
    if s["normed"] is not None:
        close(s["normed"], n, en, names(s["normed"]))


@pytest.mark.parametrize("H", [1, 7, 8, 64, 255, 256, 257, 1000, 1024, 1032, 2048, 2049, 2560, 4096, 4104, 5001,
                               8192, 8200, 16384, 16392, 32768])
def test_row_lengths(H):
    rng = np.random.default_rng(H)
    check(make(rng, 5, H), scale=0.5)
    check(make(rng, 2, H, y="f32", residual="f32", normed="f32", gate="full", wt="f32"), gate_sigmoid=True)


@pytest.mark.parametrize("y", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("residual", ["bf16", "f16", "f32"])
def test_types(y, residual):
    rng = np.random.default_rng(3)
    for normed, wt, gt in (("bf16", "f16", "bf16"), ("f16", "f32", "f16"), ("f32", "bf16", "f32")):
        check(make(rng, 9, 640, y, residual, normed, wt=wt, gate="channel", gt=gt), gate_sigmoid=True, weight_offset=1.0)
        check(make(rng, 9, 641, y, residual, normed, wt=wt, gate="token", gt=gt))


@pytest.mark.parametrize("gate", [None, "token", "channel", "full", "one"])
@pytest.mark.parametrize("sigmoid", [False, True])
def test_gates(gate, sigmoid):
    rng = np.random.default_rng(4)
    for post in (False, True):
        check(make(rng, 6, 512, gate=gate, post=post, gt="f16"), gate_sigmoid=sigmoid, scale=-0.25)


def test_parts_left_out():
    rng = np.random.default_rng(5)
    check(make(rng, 4, 768, y=None))                             # a norm alone
    check({**make(rng, 4, 768, y=None), "out": None})
    check(make(rng, 4, 768, normed=None, pre=False))             # no second norm
    check({**make(rng, 4, 768), "out": None})
    check(make(rng, 4, 768, pre=False, post=False))              # weights of 1; y as it is


@pytest.mark.parametrize("pad,shift", [(8, 0), (24, 8), (3, 0), (0, 1), (5, 3)])
def test_strides_and_alignment(pad, shift):
    rng = np.random.default_rng(6)
    s = make(rng, 11, 1024, pad=pad, shift=shift, gate="full")
    full = [t._base.clone() for t in (s["out"], s["normed"])]
    check(s)
    for t, was in zip((s["out"], s["normed"]), full):            # nothing beside the rows is written
        assert torch.equal(t._base[:, :shift], was[:, :shift])
        assert torch.equal(t._base[:, shift + 1024:], was[:, shift + 1024:])


@pytest.mark.parametrize("H", [640, 641, 9000])
def test_in_place(H):
    rng = np.random.default_rng(7)
    s = make(rng, 300, H)
    r, n, er, en = want(s)
    s["out"], s["normed"] = s["residual"], s["y"]
    moe.moe_residual_norm(**s)
    close(s["out"], r, er, "bf16")
    close(s["normed"], n, en, "bf16")


def test_many_rows_one_row_and_repeated_calls():
    rng = np.random.default_rng(8)
    s = make(rng, 5000, 384, y="f32")
    check(s)
    first = s["out"].clone(), s["normed"].clone()
    moe.moe_residual_norm(**s)
    assert torch.equal(s["out"], first[0]) and torch.equal(s["normed"], first[1])
    one = {k: v if v is None or k.endswith("weight") else v[17:18] for k, v in s.items()}
    moe.moe_residual_norm(**one)                                 # a row's result is its own
    assert torch.equal(s["normed"], first[1])


def test_extreme_rows():
    rng = np.random.default_rng(9)
    s = make(rng, 3, 512, y="f32", residual="f32", normed="f32")
    s["y"][0], s["residual"][0] = 0, 0                           # a row of zeros gives zeros
    s["y"][1] *= 1e15
    s["y"][2] *= 1e-15
    check(s)
    assert torch.all(s["normed"][0] == 0)
    s = make(rng, 2, 512)
    s["y"][0, 5] = float("nan")                                  # NaN stays in its row
    moe.moe_residual_norm(**s)
    assert torch.all(torch.isnan(s["normed"][0])) and torch.all(torch.isfinite(s["normed"][1]))
    g = make(rng, 2, 512, gate="token")
    g["gate"][:] = torch.tensor([[float("inf")], [-float("inf")]])
    check(g, gate_sigmoid=True)                                  # 1 and 0


def test_another_stream_and_a_graph():
    rng = np.random.default_rng(10)
    s = make(rng, 64, 2560, gate="channel")
    r, n, er, en = want(s)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    moe.moe_residual_norm(**s, stream=side)
    side.synchronize()
    close(s["normed"], n, en, "bf16")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        moe.moe_residual_norm(**s)
    again = make(rng, 64, 2560, gate="channel")
    for k in ("y", "residual"):
        s[k].copy_(again[k])
    graph.replay()
    torch.cuda.synchronize()
    r, n, er, en = want(s)
    close(s["out"], r, er, "bf16")
    close(s["normed"], n, en, "bf16")


@pytest.mark.parametrize("H", [512, 513, 9000, 20000])
@pytest.mark.parametrize("gate", ["token", "channel", "full"])
def test_gates_and_weights_far_from_one(H, gate):
    """y is normed before its weight, the gate and the scale meet it: none of the products on the way leaves
    the range of f32 where the result does not."""
    rng = np.random.default_rng(H)
    for y_amp, w_amp, g_amp, scale in ((1e12, 1.0, 1e30, 1.0), (1e12, 1e30, 1e-25, 1.0), (1e-12, 1.0, 1e-30, 1e30),
                                       (1e15, 1.0, 1e30, 1e-20), (1e12, 1e20, 1.0, 1e10)):
        s = make(rng, 5, H, y="f32", residual="f32", normed="f32", gate=gate, wt="f32")
        s["y"] *= y_amp / 2
        s["post_weight"] *= w_amp
        s["gate"] *= g_amp
        s["residual"] *= w_amp * g_amp * scale
        if w_amp * g_amp * scale > 1e15:                         # squares of the sum leave f32 by definition
            s["normed"] = s["pre_weight"] = None
        check(s, scale=scale, eps=1e-30)
    s = make(rng, 5, H, y="f32", residual="f32", normed="f32", gate=gate, post=False)
    s["y"] *= 1e12
    s["gate"] *= 1e30                                            # without a norm scale * gate comes first
    check(s, scale=1e-30)
