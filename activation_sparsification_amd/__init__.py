"""N:M activation pruning fused with its linear layer, and the attention, cache and norms between such layers,
for MI355X (gfx950).

The compute runs in ``libspa.so`` (hand-written HIP kernels behind a C ABI,
declared in ``include/spa.h``); this package is its thin Python binding.
"""
from ._binding import (  # noqa: F401
    EXPORTS,
    EtaCalibration,
    Fp8Weight,
    PreparedCall,
    PreparedWeight,
    PruneConfig,
    SpaError,
    decode_meta,
    encode_meta,
    eta_lookup,
    lib,
    meta_row_bytes,
    prepare_amber,
    prepare_weight,
    prefill_layout,
    prepare_weight_fp8,
    prune_nm,
    sparse_linear_decode,
    sparse_linear_decode_static,
    sparse_linear_prefill,
    sparse_linear_prefill_fp8,
    sparse_ffn_relu2_prefill,
    workspace,
    workspace_bytes,
)
# The cache, attention and norm calls are bound natively (_layer): loaded at first use, so that this package can be
# imported to build them.
_LAYER = ("KvCache", "attention_decode", "attention_prefill", "gated_residual_norm", "kv_plan", "kv_read",
          "kv_write", "new_kv_cache", "new_page_pool", "qk_norm_rope")


def __getattr__(name):
    if name not in _LAYER:
        raise AttributeError(f"module {__name__!r} has no attribute {name!r}")
    from . import _layer
    for n in _LAYER:
        globals()[n] = getattr(_layer, n)
    return globals()[name]


def __dir__():
    return sorted(set(globals()) | set(_LAYER))
