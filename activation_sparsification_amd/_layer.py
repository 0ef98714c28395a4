"""The cache, attention and norm calls: thin native binding (``_layer_native``) of the C entries in ``libspa.so``.

Tensors of several heads are ``[rows, heads, head_dim]`` with the last axis dense; the row and head strides are
free (a slice of a packed projection is passed as it is).  Forward only: a tensor that requires a gradient is refused
while gradients are recorded.  Workspaces come from torch's allocator on the current
stream for each call, so calls on several streams do not share one.  If the library or the binding is not built,
importing this module raises: there is no fallback path.
"""
from __future__ import annotations

import torch

from ._binding import SpaError, lib

lib()       # raises if libspa.so is not built
try:
    from . import _layer_native as _native
except ImportError as e:
    raise ImportError(f"{e}; run `python -m activation_sparsification_amd.build`") from e

_native._set_error(SpaError)
KvCache = _native.KvCache
kv_write = _native.kv_write
kv_read = _native.kv_read
attention_decode = _native.attention_decode
attention_prefill = _native.attention_prefill
gated_residual_norm = _native.gated_residual_norm

PAGE_TYPES = {"native": None, "fp8": torch.float8_e4m3fn, "int8": torch.int8}


def new_kv_cache(n_pages: int, page_size: int, n_heads: int, head_dim: int, dtype: torch.dtype, fmt: str = "native",
                 device="cuda") -> KvCache:
    """A zero-filled cache of ``fmt`` "native" (pages of ``dtype``), "fp8" or "int8"."""
    if fmt not in PAGE_TYPES:
        raise ValueError(f"new_kv_cache: unknown format {fmt!r}")
    shape = (n_pages, n_heads, page_size, head_dim)
    pages = [torch.zeros(shape, dtype=PAGE_TYPES[fmt] or dtype, device=device) for _ in range(2)]
    scales = [None if fmt == "native" else torch.zeros(shape[:3], device=device) for _ in range(2)]
    return KvCache(*pages, *scales)
