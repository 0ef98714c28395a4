"""ctypes binding of the cache, attention and norm entry points: argument marshalling only.

Tensors of several heads are ``[rows, heads, head_dim]`` with the last axis dense; the row and head strides are
free (a slice of a packed projection is passed as it is).  Workspaces come from torch's allocator on the current
stream for each call, so calls on several streams do not share one.
"""
from __future__ import annotations

import ctypes
import dataclasses
from typing import Optional, Tuple

import torch

from ._binding import DTYPE, _check, _Heads, _KvCache, _Norm, _ptr, _stream, lib

KV_FORMAT = {"native": 0, "fp8": 1, "int8": 2}
NORM = {"none": 0, "rms": 1, "layer": 2}
_CODES = {torch.float8_e4m3fn: 1, torch.int8: 2}


def _need(ok: bool, what: str) -> None:
    if not ok:
        raise ValueError(what)


def _heads(x: torch.Tensor, name: str) -> _Heads:
    _need(x.is_cuda, f"{name}: expected a device tensor")
    _need(x.dim() == 3, f"{name}: expected [rows, heads, head_dim]")
    row, head, last = x.stride()
    _need(last == 1 or x.shape[2] == 1, f"{name}: expected a dense last axis")
    # the stride of an axis of one element is never used, and torch leaves any number in it
    return _Heads(x.data_ptr(), row if x.shape[0] > 1 else 0, head if x.shape[1] > 1 else 0)


def _given(x: torch.Tensor, shape, dtype, device, name: str) -> torch.Tensor:
    _need(x.device == device and x.dtype == dtype and x.shape == shape and x.is_contiguous(),
          f"{name}: expected a contiguous {dtype} tensor of shape {list(shape)} on {device}")
    return x


@dataclasses.dataclass
class KvCache:
    """A paged cache of one layer: ``k`` and ``v`` are [n_pages, n_heads, page_size, head_dim].

    float16 or bfloat16 pages hold the vectors as they are; float8_e4m3fn and int8 pages hold codes, with float32
    ``k_scale`` and ``v_scale`` [n_pages, n_heads, page_size].
    """
    k: torch.Tensor
    v: torch.Tensor
    k_scale: Optional[torch.Tensor] = None
    v_scale: Optional[torch.Tensor] = None

    def __post_init__(self):
        k = self.k
        _need(k.is_cuda, "KvCache: expected device tensors")
        _need(k.dim() == 4 and k.is_contiguous(), "KvCache: k is [n_pages, n_heads, page_size, head_dim], contiguous")
        _given(self.v, k.shape, k.dtype, k.device, "KvCache.v")
        self.format = _CODES.get(k.dtype, 0)
        if self.format:
            for name in ("k_scale", "v_scale"):
                s = getattr(self, name)
                _need(s is not None, f"KvCache: {k.dtype} pages need {name}")
                _given(s, k.shape[:3], torch.float32, k.device, "KvCache." + name)
        else:
            _need(k.dtype in DTYPE, f"KvCache: pages of {k.dtype}")
            _need(self.k_scale is None and self.v_scale is None, "KvCache: scales belong to 8-bit pages")
        p, h, s, d = k.shape
        self._c = {t: _KvCache(DTYPE[t], self.format, p, s, h, d, _ptr(k), _ptr(self.v), _ptr(self.k_scale),
                               _ptr(self.v_scale)) for t in (DTYPE if self.format else (k.dtype,))}

    @property
    def n_heads(self) -> int:
        return self.k.shape[1]

    @property
    def page_size(self) -> int:
        return self.k.shape[2]

    @property
    def head_dim(self) -> int:
        return self.k.shape[3]

    def c(self, dtype: torch.dtype):
        """The C descriptor for vectors of ``dtype`` going in or out."""
        d = self._c.get(dtype)
        _need(d is not None, f"KvCache: {dtype} vectors with {self.k.dtype} pages")
        return ctypes.byref(d)


def new_kv_cache(n_pages: int, page_size: int, n_heads: int, head_dim: int, dtype: torch.dtype, fmt: str = "native",
                 device="cuda") -> KvCache:
    """A zero-filled cache of ``fmt`` "native" (pages of ``dtype``), "fp8" or "int8"."""
    _need(fmt in KV_FORMAT, f"new_kv_cache: unknown format {fmt!r}")
    shape = (n_pages, n_heads, page_size, head_dim)
    code = {"native": dtype, "fp8": torch.float8_e4m3fn, "int8": torch.int8}[fmt]
    pages = [torch.zeros(shape, dtype=code, device=device) for _ in range(2)]
    scales = [None if fmt == "native" else torch.zeros(shape[:3], device=device) for _ in range(2)]
    return KvCache(*pages, *scales)


def kv_write(k: torch.Tensor, v: torch.Tensor, slots: torch.Tensor, cache: KvCache) -> None:
    """Store the rows of ``k`` and ``v`` [t, n_heads, head_dim] at ``slots`` [t] int32 (-1: skip the row)."""
    t = k.shape[0]
    kh, vh, dev = _heads(k, "k"), _heads(v, "v"), cache.k.device
    _need(k.device == dev and v.device == dev, "kv_write: tensors on several devices")
    _need(k.shape == v.shape and k.dtype == v.dtype, "kv_write: k and v differ in shape or type")
    _need(k.shape[1] == cache.n_heads and k.shape[2] == cache.head_dim, "kv_write: the cache has other heads")
    _given(slots, (t,), torch.int32, dev, "slots")
    _check(lib().spa_kv_write(kh, vh, t, slots.data_ptr(), cache.c(k.dtype), _stream(dev)), "spa_kv_write")


def _table(page_table: torch.Tensor, n: int, dev) -> int:
    _need(page_table.dim() == 2, "page_table: expected [n_seqs, max_pages]")
    _given(page_table, (n, page_table.shape[1]), torch.int32, dev, "page_table")
    return page_table.shape[1]


def kv_read(cache: KvCache, page_table: torch.Tensor, cu_seqlens: torch.Tensor, total: int,
            k_out: Optional[torch.Tensor] = None, v_out: Optional[torch.Tensor] = None,
            dtype: Optional[torch.dtype] = None) -> Tuple[torch.Tensor, torch.Tensor]:
    """The first ``cu_seqlens[s+1] - cu_seqlens[s]`` positions of each sequence, packed: two [total, n_heads, head_dim].

    ``dtype`` is needed for 8-bit pages when no outputs are given.
    """
    dev, n = cache.k.device, page_table.shape[0]
    max_pages = _table(page_table, n, dev)
    _given(cu_seqlens, (n + 1,), torch.int32, dev, "cu_seqlens")
    if dtype is None:
        dtype = k_out.dtype if k_out is not None else None if cache.format else cache.k.dtype
    _need(dtype is not None, "kv_read: 8-bit pages need dtype or outputs")
    shape = (total, cache.n_heads, cache.head_dim)
    got = [torch.empty(shape, dtype=dtype, device=dev) if o is None else _given(o, shape, dtype, dev, name)
           for o, name in ((k_out, "k_out"), (v_out, "v_out"))]
    _check(lib().spa_kv_read(cache.c(dtype), page_table.data_ptr(), n, max_pages, cu_seqlens.data_ptr(), total,
                             got[0].data_ptr(), got[1].data_ptr(), _stream(dev)), "spa_kv_read")
    return got[0], got[1]


def _scale_of(scale: Optional[float], d: int) -> float:
    return d ** -0.5 if scale is None else float(scale)


def attention_decode(q: torch.Tensor, cache: KvCache, page_table: torch.Tensor, seq_lens: torch.Tensor,
                     scale: Optional[float] = None, want_lse: bool = False, out: Optional[torch.Tensor] = None,
                     ws: Optional[torch.Tensor] = None) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """Attention of one new token per sequence, ``q`` [n_seqs, n_q_heads, head_dim], over its cached positions.

    ``scale`` defaults to head_dim ** -0.5.  Returns ``(out [n_seqs, n_q_heads, head_dim], lse [n_seqs, n_q_heads] or
    None)``.
    """
    qh, dev = _heads(q, "q"), q.device
    n, hq, d = q.shape
    _need(cache.k.device == dev, "attention_decode: tensors on several devices")
    _need(d == cache.head_dim, "attention_decode: the cache has another head_dim")
    max_pages = _table(page_table, n, dev)
    _given(seq_lens, (n,), torch.int32, dev, "seq_lens")
    out = torch.empty((n, hq, d), dtype=q.dtype, device=dev) if out is None else _given(out, (n, hq, d), q.dtype, dev, "out")
    lse = torch.empty((n, hq), dtype=torch.float32, device=dev) if want_lse else None
    L = lib()
    if ws is None:
        ws = torch.empty(L.spa_attention_decode_workspace_bytes(n, hq, cache.n_heads, d), dtype=torch.uint8, device=dev)
    _check(L.attention_decode(qh, n, hq, cache.c(q.dtype), page_table.data_ptr(), max_pages, seq_lens.data_ptr(),
                              _scale_of(scale, d), out.data_ptr(), _ptr(lse), ws.data_ptr(), ws.numel(), _stream(dev)),
           "attention_decode")
    return out, lse


def attention_prefill(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, cu_q: torch.Tensor,
                      cu_k: Optional[torch.Tensor] = None, causal: bool = True, scale: Optional[float] = None,
                      want_lse: bool = False, out: Optional[torch.Tensor] = None,
                      ws: Optional[torch.Tensor] = None) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """Attention over packed prompts: ``q`` [tq, n_q_heads, head_dim], ``k`` and ``v`` [tk, n_kv_heads, head_dim].

    ``cu_q`` and ``cu_k`` [n_seqs + 1] int32 are the sequences' first rows and the end (``cu_k`` defaults to ``cu_q``).
    Returns ``(out [tq, n_q_heads, head_dim], lse [tq, n_q_heads] or None)``.
    """
    qh, kh, vh, dev = _heads(q, "q"), _heads(k, "k"), _heads(v, "v"), q.device
    tq, hq, d = q.shape
    _need(k.shape == v.shape and k.shape[2] == d, "attention_prefill: k and v are [tk, n_kv_heads, head_dim]")
    _need(k.dtype == q.dtype and v.dtype == q.dtype and q.dtype in DTYPE, "attention_prefill: q, k and v differ in type")
    _need(k.device == dev and v.device == dev, "attention_prefill: tensors on several devices")
    cu_k = cu_q if cu_k is None else cu_k
    n = cu_q.shape[0] - 1
    _need(n >= 0, "cu_q: expected [n_seqs + 1]")
    _given(cu_q, (n + 1,), torch.int32, dev, "cu_q")
    _given(cu_k, (n + 1,), torch.int32, dev, "cu_k")
    out = torch.empty((tq, hq, d), dtype=q.dtype, device=dev) if out is None else _given(out, (tq, hq, d), q.dtype, dev, "out")
    lse = torch.empty((tq, hq), dtype=torch.float32, device=dev) if want_lse else None
    L = lib()
    if ws is None:
        need = L.spa_attention_prefill_workspace_bytes(tq, n, hq, k.shape[1], d)
        ws = torch.empty(need, dtype=torch.uint8, device=dev) if need else None
    _check(L.attention_prefill(qh, kh, vh, DTYPE[q.dtype], tq, k.shape[0], hq, k.shape[1], d, cu_q.data_ptr(),
                               cu_k.data_ptr(), n, int(causal), _scale_of(scale, d), out.data_ptr(), _ptr(lse), _ptr(ws),
                               0 if ws is None else ws.numel(), _stream(dev)), "attention_prefill")
    return out, lse


def _norm(kind: str, weight, bias, c: int, dtype, dev, name: str) -> _Norm:
    _need(kind in NORM, f"{name}: unknown norm {kind!r}")
    for t, part in ((weight, "weight"), (bias, "bias")):
        if t is not None:
            _given(t, (c,), dtype, dev, f"{name}_{part}")
    return _Norm(NORM[kind], None if weight is None else weight.data_ptr(), None if bias is None else bias.data_ptr())


def gated_residual_norm(x: torch.Tensor, residual: Optional[torch.Tensor] = None, *, post: str = "none",
                        post_weight: Optional[torch.Tensor] = None, post_bias: Optional[torch.Tensor] = None,
                        gate: Optional[torch.Tensor] = None, scale: float = 1.0, pre: str = "rms",
                        pre_weight: Optional[torch.Tensor] = None, pre_bias: Optional[torch.Tensor] = None,
                        eps: float = 1e-5, h_out: Optional[torch.Tensor] = None,
                        y_out: Optional[torch.Tensor] = None) -> Tuple[torch.Tensor, torch.Tensor]:
    """``h = residual + scale * gate * post(x)`` and ``y = pre(h)`` for rows ``x`` [t, c]: returns ``(h, y)``.

    ``residual`` [t, c] is of x's type or float32 and gives h its type (None: zeros of x's type); ``gate`` is [c] or
    [t, c]; ``post`` and ``pre`` are "none", "rms" or "layer".  ``h_out`` may be ``residual`` and ``y_out`` may be ``x``.
    """
    _need(x.is_cuda and x.dim() == 2 and x.is_contiguous(), "x: expected a contiguous device tensor [t, c]")
    _need(x.dtype in DTYPE, f"x: type {x.dtype}")
    (t, c), dt, dev = x.shape, x.dtype, x.device
    st = dt if residual is None else residual.dtype
    _need(st in DTYPE, f"residual: type {st}")
    if residual is not None:
        _given(residual, (t, c), st, dev, "residual")
    rows = 0
    if gate is not None:
        rows = 1 if gate.dim() == 1 else t
        _given(gate, (c,) if gate.dim() == 1 else (t, c), dt, dev, "gate")
    post_n = _norm(post, post_weight, post_bias, c, dt, dev, "post")
    pre_n = _norm(pre, pre_weight, pre_bias, c, dt, dev, "pre")
    h = torch.empty((t, c), dtype=st, device=dev) if h_out is None else _given(h_out, (t, c), st, dev, "h_out")
    y = torch.empty((t, c), dtype=dt, device=dev) if y_out is None else _given(y_out, (t, c), dt, dev, "y_out")
    _check(lib().gated_residual_norm(x.data_ptr(), DTYPE[dt], t, c, _ptr(residual), DTYPE[st], post_n, _ptr(gate), rows,
                                     scale, pre_n, eps, h.data_ptr(), y.data_ptr(), _stream(dev)), "gated_residual_norm")
    return h, y
