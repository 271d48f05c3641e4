"""Serving operators around the MoE layer: thin Python binding of include/moe_serving.h.

NVFP4 matrix-vector products, the paged 8-bit key/value cache with the rotary rotation, causal
attention over it, and the verification of drafted tokens.  Each ``moe_*`` function marshals its
arguments and calls the C entry point of the same name; a non-OK status raises MoeError.
``NvFp4Linear`` keeps the buffers of one projection, as MoeLayer does for a layer.
"""
from __future__ import annotations

import ctypes
from typing import Optional

import torch

from . import _native
from ._native import MoeError, check as _check

__all__ = ["PagedKvCache", "SeqBatch", "NvFp4Linear", "kv_append_workspace_bytes",
           "attention_workspace_bytes", "linear_workspace_bytes", "verify_workspace_bytes",
           "moe_kv_append_rope_e4m3", "moe_attention_paged_e4m3", "moe_linear_nvfp4",
           "moe_verify_draft"]

_DTYPE = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2}
_I32, _F32, _U8 = torch.int32, torch.float32, torch.uint8
_current_device = torch._C._cuda_getDevice
_current_stream = torch._C._cuda_getCurrentRawStream

# These checks stand in front of calls of a few microseconds, so each reads a tensor's
# properties once and the device is compared by its index.


def _dtype(t: torch.Tensor, what: str) -> int:
    code = _DTYPE.get(t.dtype)
    if code is None:
        raise TypeError(f"{what} must be bfloat16, float16 or float32")
    return code


def _device() -> int:
    """Index of the current CUDA device, which a call's tensors must be on."""
    return _current_device()


def _queue(dev: int, stream) -> int:
    return _current_stream(dev) if stream is None else stream.cuda_stream


def _elsewhere(what: str):
    return ValueError(f"{what} must be on the current CUDA device")


def _workspace(dev: int, ws: torch.Tensor) -> int:
    """Bytes of the workspace."""
    if ws.get_device() != dev:
        raise _elsewhere("ws")
    return ws.numel() * ws.itemsize


def _need(dev: int, t: torch.Tensor, dtype: torch.dtype, shape: tuple, what: str) -> int:
    if t.get_device() != dev:
        raise _elsewhere(what)
    if t.dtype is not dtype:
        raise TypeError(f"{what} must be {dtype}")
    if t.shape != shape or not t.is_contiguous():
        raise ValueError(f"{what} must be contiguous {tuple(shape)}")
    return t.data_ptr()


def _rows(dev: int, t: torch.Tensor, dtype: torch.dtype, shape: tuple, what: str) -> int:
    """Row stride of token rows [T, heads, dim] whose heads are contiguous."""
    if t.get_device() != dev:
        raise _elsewhere(what)
    if t.dtype is not dtype:
        raise TypeError(f"{what} must be {dtype}")
    if t.shape != shape:
        raise ValueError(f"{what} must be {list(shape)}")
    T, heads, dim = shape
    s0, s1, s2 = t.stride()
    if s2 != 1 or (s1 != dim and heads > 1):
        raise ValueError(f"{what}: the heads of a token must be contiguous")
    return s0 if T > 1 else heads * dim


class PagedKvCache:
    """Paged key/value cache in E4M3 with one float32 scale per page and head.

    ``k_codes`` / ``v_codes`` are uint8 [num_pages, kv_heads, page_size, head_dim] planes (pages
    may be spaced apart, each page contiguous), ``k_scales`` / ``v_scales`` float32
    [num_pages, kv_heads].  The cache keeps references to the tensors, not copies.
    """

    def __init__(self, k_codes: torch.Tensor, v_codes: torch.Tensor, k_scales: torch.Tensor,
                 v_scales: torch.Tensor):
        for t, what in ((k_codes, "k_codes"), (v_codes, "v_codes")):
            if t.dtype != torch.uint8 or t.dim() != 4:
                raise TypeError(f"{what} must be uint8 [num_pages, kv_heads, page_size, head_dim]")
            if not t[0].is_contiguous():
                raise ValueError(f"{what}: a page must be contiguous")
        n, h, p, d = k_codes.shape
        if v_codes.shape != k_codes.shape or (n > 1 and v_codes.stride(0) != k_codes.stride(0)):
            raise ValueError("k_codes and v_codes must have the same shape and page stride")
        dev = self.dev = k_codes.get_device()
        if dev < 0 or v_codes.get_device() != dev:
            raise ValueError("the cache's planes must be on one CUDA device")
        _need(dev, k_scales, _F32, (n, h), "k_scales")
        _need(dev, v_scales, _F32, (n, h), "v_scales")
        self.k_codes, self.v_codes, self.k_scales, self.v_scales = k_codes, v_codes, k_scales, v_scales
        self.num_pages, self.kv_heads, self.page_size, self.head_dim = n, h, p, d
        stride = k_codes.stride(0) if n > 1 else h * p * d
        self._c = _native.KvCache(k_codes.data_ptr(), v_codes.data_ptr(), k_scales.data_ptr(),
                                  v_scales.data_ptr(), n, h, p, d, stride)
        self._ref = ctypes.byref(self._c)

    @classmethod
    def allocate(cls, num_pages: int, kv_heads: int, page_size: int, head_dim: int,
                 device="cuda") -> "PagedKvCache":
        """An empty cache (codes 0, scales 1)."""
        shape = (num_pages, kv_heads, page_size, head_dim)
        codes = torch.zeros(2, *shape, dtype=torch.uint8, device=device)
        scales = torch.ones(2, num_pages, kv_heads, dtype=torch.float32, device=device)
        return cls(codes[0], codes[1], scales[0], scales[1])

    def nbytes(self) -> int:
        return 2 * self.k_codes.numel() + 8 * self.k_scales.numel()


class SeqBatch:
    """A ragged batch: ``q_offsets`` int32 [B+1] (token rows of each sequence's new tokens),
    ``seq_lens`` int32 [B] (tokens of each sequence, the new ones counted) and ``page_table``
    int32 [B, max_pages].  The arrays are read when a call runs, so their contents may change
    between calls (or graph replays)."""

    def __init__(self, q_offsets: torch.Tensor, seq_lens: torch.Tensor, page_table: torch.Tensor):
        if page_table.dim() != 2 or page_table.dtype != torch.int32 or \
                (page_table.shape[1] > 1 and page_table.stride(1) != 1):
            raise TypeError("page_table must be int32 [B, max_pages] with contiguous rows")
        B, cols = page_table.shape
        dev = self.dev = page_table.get_device()
        if dev < 0:
            raise ValueError("the batch's arrays must be on a CUDA device")
        _need(dev, seq_lens, _I32, (B,), "seq_lens")
        _need(dev, q_offsets, _I32, (B + 1,), "q_offsets")
        self.q_offsets, self.seq_lens, self.page_table = q_offsets, seq_lens, page_table
        self.B, self.max_pages = B, cols
        stride = page_table.stride(0) if B > 1 else cols
        self._c = _native.SeqBatch(q_offsets.data_ptr(), seq_lens.data_ptr(), page_table.data_ptr(),
                                   B, cols, stride)
        self._ref = ctypes.byref(self._c)


def kv_append_workspace_bytes() -> int:
    return int(_native.load().moe_kv_append_workspace_bytes())


def attention_workspace_bytes(q_heads: int, kv_heads: int, head_dim: int) -> int:
    return int(_native.load().moe_attention_workspace_bytes(q_heads, kv_heads, head_dim))


def linear_workspace_bytes(T: int, N: int, K: int) -> int:
    return int(_native.load().moe_linear_workspace_bytes(T, N, K))


def verify_workspace_bytes(B: int, V: int) -> int:
    return int(_native.load().moe_verify_workspace_bytes(B, V))


def moe_kv_append_rope_e4m3(cache: PagedKvCache, batch: SeqBatch, k: torch.Tensor, v: torch.Tensor,
                            cos: Optional[torch.Tensor], sin: Optional[torch.Tensor],
                            ws: torch.Tensor, q: Optional[torch.Tensor] = None,
                            q_out: Optional[torch.Tensor] = None,
                            positions: Optional[torch.Tensor] = None, interleaved: bool = False,
                            stream=None) -> None:
    """Append k, v [T, kv_heads, head_dim] to the cache, keys rotated by cos/sin [max_pos,
    rotary_dim/2] (None: not rotated), and write the rotated q [T, q_heads, head_dim] to q_out
    (q itself when None)."""
    dev = _device()
    if cache.dev != dev or batch.dev != dev:
        raise _elsewhere("cache and batch")
    T, h, d, dt = k.shape[0], cache.kv_heads, cache.head_dim, k.dtype
    ks, vs = _rows(dev, k, dt, (T, h, d), "k"), _rows(dev, v, dt, (T, h, d), "v")
    qh = qs = qos = 0
    qp = qop = None
    if q is not None:
        q_out = q if q_out is None else q_out
        qh = q.shape[1]
        qs, qos = _rows(dev, q, dt, (T, qh, d), "q"), _rows(dev, q_out, dt, (T, qh, d), "q_out")
        qp, qop = q.data_ptr(), q_out.data_ptr()
    max_pos = rotary = 0
    cp = sp = pp = None
    if cos is not None or sin is not None:
        if cos is None or sin is None:
            raise ValueError("pass both cos and sin, or neither")
        max_pos, half = shape = cos.shape
        rotary = 2 * half
        cp, sp = _need(dev, cos, _F32, shape, "cos"), _need(dev, sin, _F32, shape, "sin")
    if positions is not None:
        pp = _need(dev, positions, _I32, (T,), "positions")
    _check(_native.load().moe_kv_append_rope_e4m3(
        cache._ref, batch._ref, T, k.data_ptr(), ks, v.data_ptr(), vs, qp, qs, qop, qos, qh,
        _dtype(k, "k"), cp, sp, max_pos, rotary, 1 if interleaved else 0, pp, ws.data_ptr(),
        _workspace(dev, ws), _queue(dev, stream)), "moe_kv_append_rope_e4m3")


def moe_attention_paged_e4m3(q: torch.Tensor, cache: PagedKvCache, batch: SeqBatch,
                             out: torch.Tensor, ws: torch.Tensor, scale: Optional[float] = None,
                             window: int = 0, lse: Optional[torch.Tensor] = None,
                             stream=None) -> None:
    """Causal attention of the new tokens q [T, q_heads, head_dim] over the cache into out (same
    shape and type); scale defaults to head_dim**-0.5; lse float32 [T, q_heads] if given."""
    dev = _device()
    if cache.dev != dev or batch.dev != dev:
        raise _elsewhere("cache and batch")
    d, shape, dt = cache.head_dim, q.shape, q.dtype
    if len(shape) != 3 or shape[2] != d:
        raise ValueError(f"q must be [tokens, heads, {d}]")
    T, qh, _ = shape
    qs, os_ = _rows(dev, q, dt, shape, "q"), _rows(dev, out, dt, shape, "out")
    lp = None if lse is None else _need(dev, lse, _F32, (T, qh), "lse")
    _check(_native.load().moe_attention_paged_e4m3(
        q.data_ptr(), qs, T, qh, _dtype(q, "q"), cache._ref, batch._ref,
        d ** -0.5 if scale is None else scale, window, out.data_ptr(), os_, lp, ws.data_ptr(),
        _workspace(dev, ws), _queue(dev, stream)), "moe_attention_paged_e4m3")


def moe_linear_nvfp4(x: torch.Tensor, bank, y: torch.Tensor, ws: torch.Tensor, stream=None) -> None:
    """y [T, N] = x [T, K] W^T with W an NvFp4Bank of one expert (N rows of K weights)."""
    dev = _device()
    if x.get_device() != dev or y.get_device() != dev or bank.codes.get_device() != dev:
        raise _elsewhere("x, y and the bank")
    shape, N = x.shape, bank.rows
    if len(shape) != 2 or shape[1] != bank.in_f or y.shape != (shape[0], N):
        raise ValueError("x must be [T, in_f] and y [T, rows] of the bank")
    T, K = shape
    (xs, x1), (ys, y1) = x.stride(), y.stride()
    if x1 != 1 or (y1 != 1 and N > 1):
        raise ValueError("the rows of x and y must be contiguous")
    _check(_native.load().moe_linear_nvfp4(
        x.data_ptr(), xs if T > 1 else K, _dtype(x, "x"), T, ctypes.byref(bank._c), y.data_ptr(),
        ys if T > 1 else N, _dtype(y, "y"), ws.data_ptr(), _workspace(dev, ws),
        _queue(dev, stream)), "moe_linear_nvfp4")


def moe_verify_draft(draft_ids: torch.Tensor, target_probs: torch.Tensor, u_accept: torch.Tensor,
                     u_sample: torch.Tensor, out_ids: torch.Tensor, n_accepted: torch.Tensor,
                     ws: torch.Tensor, draft_probs: Optional[torch.Tensor] = None,
                     n_draft: Optional[torch.Tensor] = None, stream=None) -> None:
    """Accept or refuse draft_ids int32 [B, n] against target_probs [B, n+1, V] (and draft_probs
    [B, n, V]) with u_accept [B, n] and u_sample [B] in [0, 1); out_ids int32 [B, n+1] gets the
    accepted ids, the drawn one, then -1, and n_accepted int32 [B] their number."""
    dev = _device()
    B, n = draft_ids.shape
    V, dt = target_probs.shape[2], target_probs.dtype
    ts = _prob_rows(dev, target_probs, dt, (B, n + 1, V), "target_probs")
    ds, dp = 0, None
    if draft_probs is not None:
        ds = _prob_rows(dev, draft_probs, dt, (B, n, V), "draft_probs")
        dp = draft_probs.data_ptr()
    np_ = None if n_draft is None else _need(dev, n_draft, _I32, (B,), "n_draft")
    _check(_native.load().moe_verify_draft(
        _need(dev, draft_ids, _I32, (B, n), "draft_ids"), np_, B, n, V, target_probs.data_ptr(), ts,
        dp, ds, _dtype(target_probs, "target_probs"),
        _need(dev, u_accept, _F32, (B, n), "u_accept"),
        _need(dev, u_sample, _F32, (B,), "u_sample"),
        _need(dev, out_ids, _I32, (B, n + 1), "out_ids"),
        _need(dev, n_accepted, _I32, (B,), "n_accepted"), ws.data_ptr(), _workspace(dev, ws),
        _queue(dev, stream)), "moe_verify_draft")


def _prob_rows(dev: int, t: torch.Tensor, dtype: torch.dtype, shape: tuple, what: str) -> int:
    """Stride between the rows of [B, rows, V], which must be the same across sequences."""
    if t.get_device() != dev:
        raise _elsewhere(what)
    if t.dtype is not dtype:
        raise TypeError(f"{what} must be {dtype}")
    if t.shape != shape:
        raise ValueError(f"{what} must be {list(shape)}")
    B, rows, V = shape
    sb, sr, sv = t.stride()
    if sv != 1 and V > 1:
        raise ValueError(f"{what}: a row must be contiguous")
    stride = sr if rows > 1 else sb if B > 1 else V
    if B > 1 and rows > 0 and sb != rows * stride:
        raise ValueError(f"{what}: rows must be evenly spaced over sequences")
    return stride


class NvFp4Linear:
    """One projection with NVFP4 weights: the bank (one expert) plus its buffers, allocated once
    and reused, so repeated calls allocate nothing.

    Buffers are kept per stream and for powers of two of tokens (calls of any sizes up to T keep at
    most four times what one of T needs).  The rows that ``forward`` returns are the first of such
    a buffer: the stream's next call whose tokens round up to the same power of two overwrites
    them.  A call that is captured in a graph uses the buffers of an earlier call of its size, if
    there was one; replays must not overlap that stream's calls."""

    def __init__(self, bank, out_dtype: torch.dtype = torch.bfloat16):
        if bank.E != 1:
            raise ValueError("a linear layer's bank has one expert")
        self.bank, self.out_dtype = bank, out_dtype
        self._kept = {}                          # by (tokens, a power of two; stream handle)
        self._bufs = {}                          # their first rows by (tokens, stream handle)

    def buffers(self, T: int, stream=None) -> dict:
        key = T, _queue(_device(), stream)
        return self._bufs.get(key) or self._new_buffers(key, stream)

    def _new_buffers(self, key: tuple, stream) -> dict:
        T, handle = key
        if linear_workspace_bytes(T, self.bank.rows, self.bank.in_f) == 0:
            raise MoeError(2, "linear_workspace_bytes")
        most = 1 << (T - 1).bit_length()
        # on the call's stream: its kernels come behind the fill, and behind whatever used the
        # memory before
        with torch.cuda.stream(stream):
            kept = self._kept.get((most, handle))
            if kept is None and torch.cuda.is_current_stream_capturing():
                for (m, _), other in self._kept.items():
                    if m == most:                # lent to the capture only
                        return {"ws": other["ws"], "y": other["y"][:T]}
            if kept is None:
                n = linear_workspace_bytes(most, self.bank.rows, self.bank.in_f)
                dev = self.bank.codes.device
                kept = self._kept[most, handle] = {
                    "ws": torch.zeros(n, dtype=torch.uint8, device=dev),
                    "y": torch.empty(most, self.bank.rows, dtype=self.out_dtype, device=dev),
                }
        b = self._bufs[key] = {"ws": kept["ws"], "y": kept["y"][:T]}
        return b

    def forward(self, x: torch.Tensor, stream=None) -> torch.Tensor:
        b = self.buffers(x.shape[0], stream)
        moe_linear_nvfp4(x, self.bank, b["y"], b["ws"], stream)
        return b["y"]
