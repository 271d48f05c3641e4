"""moe_linear_nvfp4 against the float64 oracle, within the bound of a float32 accumulation plus
the rounding of the output type."""
import numpy as np
import pytest
import torch

import nvfp4_grouped_gemm_gb300 as moe
from oracle import serving as oracle
from oracle.nvfp4 import dequant
from serving_util import DT, activations, zeros_ws

pytestmark = pytest.mark.gpu
# half a unit in the last place of 8, 11 and 24 significant bits, and half the least subnormal
ROUND = {"bf16": (2.0 ** -8, 2.0 ** -134), "f16": (2.0 ** -11, 2.0 ** -25),
         "f32": (2.0 ** -24, 2.0 ** -150)}


def bank_of(rng, N, K, alpha=None):
    codes = rng.integers(0, 256, (1, N, K // 2), dtype=np.uint8)
    scales = rng.integers(0x00, 0x40, (1, N, K // 16), dtype=np.uint8)
    w = dequant(codes[0], scales[0]) * (1 if alpha is None else np.float64(np.float32(alpha)))
    a = None if alpha is None else torch.tensor([alpha], dtype=torch.float32).cuda()
    return moe.NvFp4Bank(torch.from_numpy(codes).cuda(), torch.from_numpy(scales).cuda(), a), w


def check(rng, T, N, K, xd, yd, alpha=None, amp=1.0, strided=False):
    bank, w = bank_of(rng, N, K, alpha)
    x = activations(rng, (T, K), xd, amp)
    if amp == 1.0 and T > 1:
        x[T // 2] *= 2.0 ** -10
    want, tol = oracle.linear(x.double().numpy(), w)
    rel, floor = ROUND[yd]
    tol = tol + rel * (np.abs(want) + tol) + floor
    if strided:
        xs = torch.zeros(T, K + 64, dtype=DT[xd], device="cuda")
        xs[:, 32:32 + K] = x.cuda()
        x_dev = xs[:, 32:32 + K]
        y = torch.full((T, N + 13), 7.0, dtype=DT[yd], device="cuda")
        y_dev = y[:, 5:5 + N]
    else:
        x_dev, y_dev = x.cuda(), torch.full((T, N), float("nan"), dtype=DT[yd], device="cuda")
    ws = zeros_ws(moe.linear_workspace_bytes(T, N, K))
    for _ in range(2):                                  # the workspace serves another call
        moe.moe_linear_nvfp4(x_dev, bank, y_dev, ws)
    got = y_dev.double().cpu().numpy()
    assert moe.get_device_error(ws) == 0
    assert np.all(np.abs(got - want) <= tol), float(np.max(np.abs(got - want) / tol))
    if strided:
        assert (y[:, :5] == 7).all() and (y[:, 5 + N:] == 7).all()
    return y_dev


@pytest.mark.parametrize("T,N,K,xd,yd", [
    (1, 1, 32, "bf16", "f32"), (1, 17, 64, "f16", "f16"), (2, 15, 96, "bf16", "bf16"),
    (3, 640, 2560, "bf16", "f32"), (8, 333, 640, "f16", "f32"), (9, 200, 352, "bf16", "f32"),
    (1, 5120, 2560, "bf16", "bf16"), (16, 1027, 4096, "bf16", "f32"), (31, 65, 1056, "f16", "f16"),
    (33, 100, 320, "bf16", "f32"), (1, 4099, 4096, "f16", "f32"), (7, 48, 65536, "bf16", "f32"),
    (128, 129, 256, "bf16", "f32"), (1, 40000, 608, "bf16", "f32"), (5, 2561, 640, "bf16", "f32"),
    (24, 3000, 8192, "bf16", "bf16"), (4, 16, 16384, "f16", "f32")])
def test_sizes_and_types(T, N, K, xd, yd):
    check(np.random.default_rng(T + N + K), T, N, K, xd, yd)


def test_alpha_strides_and_magnitudes():
    rng = np.random.default_rng(5)
    check(rng, 4, 130, 512, "bf16", "f32", alpha=0.00037)
    check(rng, 3, 131, 512, "bf16", "f32", strided=True)
    check(rng, 12, 77, 544, "f16", "bf16", strided=True)
    check(rng, 2, 64, 512, "bf16", "f32", amp=1e30)
    check(rng, 2, 64, 512, "bf16", "f32", amp=1e-30)


def test_infinities_and_nan_stay_in_their_rows():
    rng = np.random.default_rng(6)
    bank, w = bank_of(rng, 70, 256)
    x = activations(rng, (3, 256), "bf16")
    clean = x.clone()
    x[1, 5] = float("nan")
    ws = zeros_ws(moe.linear_workspace_bytes(3, 70, 256))
    a, b = torch.empty(3, 70, device="cuda"), torch.empty(3, 70, device="cuda")
    moe.moe_linear_nvfp4(clean.cuda(), bank, a, ws)
    moe.moe_linear_nvfp4(x.cuda(), bank, b, ws)
    assert torch.equal(a[0], b[0]) and torch.equal(a[2], b[2])
    assert torch.isnan(b[1]).all()


def test_the_layer_object_keeps_its_buffers():
    rng = np.random.default_rng(7)
    bank, w = bank_of(rng, 96, 128)
    lin = moe.NvFp4Linear(bank, torch.float32)
    x = activations(rng, (2, 128), "bf16").cuda()
    y = lin.forward(x)
    want, tol = oracle.linear(x.double().cpu().numpy(), w)
    assert np.all(np.abs(y.double().cpu().numpy() - want) <= tol)
    assert lin.forward(x).data_ptr() == y.data_ptr()


def busy():
    """Some tens of milliseconds of work on the current stream."""
    a = torch.ones(8192, 8192, dtype=torch.bfloat16, device="cuda")
    for _ in range(30):
        a @ a


def test_the_layer_object_s_buffers_belong_to_the_call_s_stream():
    """A call on another stream than the current one: neither the zero fill of a new workspace nor
    memory that the current stream still writes may come behind it."""
    rng = np.random.default_rng(8)
    T, N, K = 16, 3001, 2048
    bank, w = bank_of(rng, N, K)
    x = activations(rng, (T, K), "bf16")
    want, tol = oracle.linear(x.double().numpy(), w)
    tol = tol + ROUND["f32"][0] * (np.abs(want) + tol)
    x, side = x.cuda(), torch.cuda.Stream()
    ws_bytes = moe.linear_workspace_bytes(T, N, K)
    torch.cuda.synchronize()
    for _ in range(2):
        # blocks of the sizes the object asks for, last written by work that is still queued
        busy()
        for rows in (16, 32):
            y = torch.full((rows, N), 7.0, device="cuda")
            del y
        for n in (ws_bytes, moe.linear_workspace_bytes(32, N, K)):
            ws = torch.full((n,), 255, dtype=torch.uint8, device="cuda")
            del ws
        lin = moe.NvFp4Linear(bank, torch.float32)
        y = lin.forward(x, stream=side)
        torch.cuda.synchronize()
        assert np.all(np.abs(y.double().cpu().numpy() - want) <= tol)


def test_the_layer_object_s_calls_on_two_streams_do_not_share_buffers():
    rng = np.random.default_rng(9)
    bank, w = bank_of(rng, 500, 4096)
    lin = moe.NvFp4Linear(bank, torch.float32)
    xs = [activations(rng, (16, 4096), "bf16") for _ in range(2)]
    wants = [oracle.linear(x.double().numpy(), w) for x in xs]
    xs, streams = [x.cuda() for x in xs], [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(20):
        ys = [lin.forward(x, stream=s) for x, s in zip(xs, streams)]
    torch.cuda.synchronize()
    assert ys[0].data_ptr() != ys[1].data_ptr()
    for y, (want, tol) in zip(ys, wants):
        assert np.all(np.abs(y.double().cpu().numpy() - want) <= tol + 2.0 ** -24 * (np.abs(want) + tol))


def test_the_layer_object_captures_with_the_buffers_of_the_call_before():
    """A warm-up call's buffers serve the capture, and calls of other sizes leave them alone."""
    rng = np.random.default_rng(10)
    bank, w = bank_of(rng, 300, 1024)
    lin = moe.NvFp4Linear(bank, torch.float32)
    x = activations(rng, (3, 1024), "bf16").cuda()
    warm = lin.forward(x)
    first = warm.clone()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = lin.forward(x)
    assert y.data_ptr() == warm.data_ptr()
    for T in (40, 1, 200):                       # buffers of other sizes; the graph's stay its own
        lin.forward(activations(rng, (T, 1024), "bf16").cuda())
    y.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(y, first)


def test_the_layer_object_s_memory_follows_the_largest_call():
    """Calls of every size up to T keep no more than a few times the largest one's buffers."""
    rng = np.random.default_rng(11)
    bank, w = bank_of(rng, 20011, 512)
    lin = moe.NvFp4Linear(bank, torch.float32)
    xs = activations(rng, (96, 512), "bf16")
    want, tol = oracle.linear(xs.double().numpy(), w)
    tol = tol + 2.0 ** -24 * (np.abs(want) + tol)
    xs = xs.cuda()
    largest = 128 * 20011 * 4 + moe.linear_workspace_bytes(128, 20011, 512)
    torch.cuda.synchronize()
    before = torch.cuda.memory_allocated()
    for T in range(1, 97):
        y = lin.forward(xs[:T])
        assert y.shape == (T, 20011)
    assert torch.cuda.memory_allocated() - before <= 2.5 * largest
    for T in (96, 5, 64, 1):
        y = lin.forward(xs[:T])
        assert np.all(np.abs(y.double().cpu().numpy() - want[:T]) <= tol[:T])


@pytest.mark.parametrize("T,N,K,xd", [(513, 40, 4096, "bf16"), (600, 33, 1024, "bf16"),
                                      (515, 20, 8192, "f16"), (513, 17, 16384, "bf16"),
                                      (514, 18, 32768, "bf16"), (513, 16, 65536, "bf16"),
                                      (512, 21, 1056, "bf16"), (700, 50, 352, "f16")])
def test_more_tokens_than_are_prepared_at_once(T, N, K, xd):
    check(np.random.default_rng(T + N + K), T, N, K, xd, "f32")
