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
from ._native import MoeError, check as _check, ptr as _ptr, stream as _stream

__all__ = ["PagedKvCache", "SeqBatch", "NvFp4Linear", "kv_append_workspace_bytes",
           "attention_workspace_bytes", "linear_workspace_bytes", "verify_workspace_bytes",
           "moe_kv_append_rope_e4m3", "moe_attention_paged_e4m3", "moe_linear_nvfp4",
           "moe_verify_draft"]

_DTYPE = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2}


def _dtype(t: torch.Tensor, what: str) -> int:
    code = _DTYPE.get(t.dtype)
    if code is None:
        raise TypeError(f"{what} must be bfloat16, float16 or float32")
    return code


def _on(dev: torch.device, t: torch.Tensor, what: str) -> None:
    if t.device != dev or not t.is_cuda:
        raise ValueError(f"{what} must be a CUDA tensor on the call's device")


def _need(dev: torch.device, t: torch.Tensor, dtype: torch.dtype, shape, what: str) -> None:
    _on(dev, t, what)
    if t.dtype != dtype:
        raise TypeError(f"{what} must be {dtype}")
    if t.shape != shape or not t.is_contiguous():
        raise ValueError(f"{what} must be contiguous {tuple(shape)}")


def _rows(dev: torch.device, t: torch.Tensor, heads: int, dim: int, what: str) -> int:
    """Row stride of token rows [T, heads, dim] whose heads are contiguous."""
    _on(dev, t, what)
    if t.dim() != 3 or t.shape[1] != heads or t.shape[2] != dim:
        raise ValueError(f"{what} must be [tokens, {heads}, {dim}]")
    if t.stride(2) != 1 or (heads > 1 and t.stride(1) != dim):
        raise ValueError(f"{what}: the heads of a token must be contiguous")
    return t.stride(0) if t.shape[0] > 1 else heads * dim


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
        self.device = k_codes.device
        _on(self.device, k_codes, "k_codes")
        _on(self.device, v_codes, "v_codes")
        _need(self.device, k_scales, torch.float32, (n, h), "k_scales")
        _need(self.device, v_scales, torch.float32, (n, h), "v_scales")
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
        self.device = page_table.device
        _on(self.device, page_table, "page_table")
        _need(self.device, seq_lens, torch.int32, (B,), "seq_lens")
        _need(self.device, q_offsets, torch.int32, (B + 1,), "q_offsets")
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
    T, h, d, dev = k.shape[0], cache.kv_heads, cache.head_dim, cache.device
    ks, vs = _rows(dev, k, h, d, "k"), _rows(dev, v, h, d, "v")
    _on(dev, ws, "ws")
    _on(dev, batch.page_table, "batch")
    if v.shape[0] != T or v.dtype != k.dtype:
        raise ValueError("k and v must have the same tokens and type")
    qh = qs = qos = 0
    if q is not None:
        q_out = q if q_out is None else q_out
        qh = q.shape[1]
        qs, qos = _rows(dev, q, qh, d, "q"), _rows(dev, q_out, qh, d, "q_out")
        if q.shape[0] != T or q_out.shape[0] != T or q.dtype != k.dtype or q_out.dtype != k.dtype:
            raise ValueError("q and q_out must have k's tokens and type")
    max_pos = rotary = 0
    if cos is not None or sin is not None:
        if cos is None or sin is None:
            raise ValueError("pass both cos and sin, or neither")
        max_pos, rotary = cos.shape[0], 2 * cos.shape[1]
        _need(dev, cos, torch.float32, (max_pos, rotary // 2), "cos")
        _need(dev, sin, torch.float32, (max_pos, rotary // 2), "sin")
    if positions is not None:
        _need(dev, positions, torch.int32, (T,), "positions")
    _check(_native.load().moe_kv_append_rope_e4m3(
        cache._ref, batch._ref, T, k.data_ptr(), ks, v.data_ptr(), vs, _ptr(q), qs,
        _ptr(q_out) if q is not None else None, qos, qh, _dtype(k, "k"), _ptr(cos), _ptr(sin),
        max_pos, rotary, 1 if interleaved else 0, _ptr(positions), ws.data_ptr(), ws.nbytes,
        _stream(stream)), "moe_kv_append_rope_e4m3")


def moe_attention_paged_e4m3(q: torch.Tensor, cache: PagedKvCache, batch: SeqBatch,
                             out: torch.Tensor, ws: torch.Tensor, scale: Optional[float] = None,
                             window: int = 0, lse: Optional[torch.Tensor] = None,
                             stream=None) -> None:
    """Causal attention of the new tokens q [T, q_heads, head_dim] over the cache into out (same
    shape and type); scale defaults to head_dim**-0.5; lse float32 [T, q_heads] if given."""
    d, dev = cache.head_dim, cache.device
    T, qh = q.shape[0], q.shape[1]
    qs, os_ = _rows(dev, q, qh, d, "q"), _rows(dev, out, qh, d, "out")
    _on(dev, ws, "ws")
    _on(dev, batch.page_table, "batch")
    if out.shape[0] != T or out.dtype != q.dtype:
        raise ValueError("out must have q's shape and type")
    if lse is not None:
        _need(dev, lse, torch.float32, (T, qh), "lse")
    _check(_native.load().moe_attention_paged_e4m3(
        q.data_ptr(), qs, T, qh, _dtype(q, "q"), cache._ref, batch._ref,
        d ** -0.5 if scale is None else scale, window, out.data_ptr(), os_, _ptr(lse),
        ws.data_ptr(), ws.nbytes, _stream(stream)), "moe_attention_paged_e4m3")


def moe_linear_nvfp4(x: torch.Tensor, bank, y: torch.Tensor, ws: torch.Tensor, stream=None) -> None:
    """y [T, N] = x [T, K] W^T with W an NvFp4Bank of one expert (N rows of K weights)."""
    if x.dim() != 2 or y.dim() != 2 or x.shape[1] != bank.in_f or \
            y.shape[0] != x.shape[0] or y.shape[1] != bank.rows:
        raise ValueError("x must be [T, in_f] and y [T, rows] of the bank")
    if x.stride(1) != 1 or (y.shape[1] > 1 and y.stride(1) != 1):
        raise ValueError("the rows of x and y must be contiguous")
    T, dev = x.shape[0], bank.codes.device
    _on(dev, x, "x")
    _on(dev, y, "y")
    _on(dev, ws, "ws")
    _check(_native.load().moe_linear_nvfp4(
        x.data_ptr(), x.stride(0) if T > 1 else bank.in_f, _dtype(x, "x"), T,
        ctypes.byref(bank._c), y.data_ptr(), y.stride(0) if T > 1 else bank.rows, _dtype(y, "y"),
        ws.data_ptr(), ws.nbytes, _stream(stream)), "moe_linear_nvfp4")


def moe_verify_draft(draft_ids: torch.Tensor, target_probs: torch.Tensor, u_accept: torch.Tensor,
                     u_sample: torch.Tensor, out_ids: torch.Tensor, n_accepted: torch.Tensor,
                     ws: torch.Tensor, draft_probs: Optional[torch.Tensor] = None,
                     n_draft: Optional[torch.Tensor] = None, stream=None) -> None:
    """Accept or refuse draft_ids int32 [B, n] against target_probs [B, n+1, V] (and draft_probs
    [B, n, V]) with u_accept [B, n] and u_sample [B] in [0, 1); out_ids int32 [B, n+1] gets the
    accepted ids, the drawn one, then -1, and n_accepted int32 [B] their number."""
    B, n = draft_ids.shape
    V = target_probs.shape[2]
    ts = _prob_rows(target_probs, B, n + 1, V, "target_probs")
    ds = 0
    if draft_probs is not None:
        ds = _prob_rows(draft_probs, B, n, V, "draft_probs")
        _on(target_probs.device, draft_probs, "draft_probs")
        if draft_probs.dtype != target_probs.dtype:
            raise TypeError("draft_probs must have target_probs' type")
    i32, f32, dev = torch.int32, torch.float32, target_probs.device
    _on(dev, target_probs, "target_probs")
    _on(dev, ws, "ws")
    _need(dev, draft_ids, i32, (B, n), "draft_ids")
    _need(dev, u_accept, f32, (B, n), "u_accept")
    _need(dev, u_sample, f32, (B,), "u_sample")
    _need(dev, out_ids, i32, (B, n + 1), "out_ids")
    _need(dev, n_accepted, i32, (B,), "n_accepted")
    if n_draft is not None:
        _need(dev, n_draft, i32, (B,), "n_draft")
    _check(_native.load().moe_verify_draft(
        draft_ids.data_ptr(), _ptr(n_draft), B, n, V, target_probs.data_ptr(), ts,
        _ptr(draft_probs), ds, _dtype(target_probs, "target_probs"), u_accept.data_ptr(),
        u_sample.data_ptr(), out_ids.data_ptr(), n_accepted.data_ptr(), ws.data_ptr(), ws.nbytes,
        _stream(stream)), "moe_verify_draft")


def _prob_rows(t: torch.Tensor, B: int, rows: int, V: int, what: str) -> int:
    """Stride between the rows of [B, rows, V], which must be the same across sequences."""
    if t.dim() != 3 or t.shape[0] != B or t.shape[1] != rows or t.shape[2] != V:
        raise ValueError(f"{what} must be [{B}, {rows}, {V}]")
    sb, sr, sv = t.stride()
    if V > 1 and sv != 1:
        raise ValueError(f"{what}: a row must be contiguous")
    stride = sr if rows > 1 else sb if B > 1 else V
    if B > 1 and rows > 0 and sb != rows * stride:
        raise ValueError(f"{what}: rows must be evenly spaced over sequences")
    return stride


class NvFp4Linear:
    """One projection with NVFP4 weights: the bank (one expert) plus its buffers per token count,
    allocated once and reused, so repeated calls allocate nothing."""

    def __init__(self, bank, out_dtype: torch.dtype = torch.bfloat16):
        if bank.E != 1:
            raise ValueError("a linear layer's bank has one expert")
        self.bank, self.out_dtype = bank, out_dtype
        self._bufs = {}

    def buffers(self, T: int) -> dict:
        if T not in self._bufs:
            dev = self.bank.codes.device
            n = linear_workspace_bytes(T, self.bank.rows, self.bank.in_f)
            if n == 0:
                raise MoeError(2, "linear_workspace_bytes")
            self._bufs[T] = {
                "ws": torch.zeros(n, dtype=torch.uint8, device=dev),
                "y": torch.empty(T, self.bank.rows, dtype=self.out_dtype, device=dev),
            }
        return self._bufs[T]

    def forward(self, x: torch.Tensor, stream=None) -> torch.Tensor:
        b = self.buffers(x.shape[0])
        moe_linear_nvfp4(x, self.bank, b["y"], b["ws"], stream)
        return b["y"]
