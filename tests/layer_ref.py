"""Plain 64-bit forms of the cache, attention and norm operators, and the error bounds their tests use.

Bounds are sums of the roundings the library's definition allows, evaluated on the reference's own numbers:
with u the unit roundoff of the 16-bit type (2^-8 bfloat16, 2^-11 float16)

* an attention output: u |o| for its own rounding, u sum p |v| for the 16-bit rounding of each softmax weight, and
  the float32 errors of the score (2 ds on each weight, ds = (d + 8) 2^-24 scale sum |q k|, plus 2^-18 for exp2) times
  sum p |v|; float16 weights below 2^-14 are rounded absolutely, 2^-25 each against a sum of at least 1;
* a log-sum-exp: ds and 2^-18 of its size plus 1;
* a norm: its own rounding, and 2^-17 of the size of its terms for the float32 sums and the root.
"""
import math

import torch

U = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}
TOP = {"fp8": 448.0, "int8": 127.0}
CODE = {"fp8": torch.float8_e4m3fn, "int8": torch.int8}


def f32(x64):
    """The nearest float32, as float64."""
    return x64.float().double()


def e4m3(y):
    """The nearest e4m3 value (ties to even) of float64 numbers up to 448, as float64."""
    step = torch.exp2(torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6))) - 3)
    return (y / step).round() * step


def quantise(x, fmt):
    """Code values and scales (float64 holding float32 numbers) of vectors along the last axis."""
    x = x.double()
    a = x.abs().amax(-1)
    live = a >= 2.0 ** -100
    safe = torch.where(live, a, torch.ones_like(a))
    scale = torch.where(live, f32(safe / TOP[fmt]), torch.zeros_like(a))
    inv = torch.where(live, f32(TOP[fmt] / safe), torch.zeros_like(a))
    y = f32(x * inv[..., None])
    return (e4m3(y) if fmt == "fp8" else y.round()), scale


def attention(q, k, v, scale, visible, p_floor=0.0):
    """One sequence: q [lq, hq, d], k and v [lk, hkv, d] float64, visible [lq, lk] bool.

    Returns out, lse and their bounds.  p_floor: the absolute rounding of one weight times its value, for float16.
    """
    lq, hq, d = q.shape
    lk, hkv = k.shape[:2]
    out = torch.zeros_like(q)
    lse = torch.full((lq, hq), -math.inf, dtype=torch.float64, device=q.device)
    weight, ds = torch.zeros_like(q), torch.zeros_like(lse)
    if lk == 0 or lq == 0:
        return out, lse, weight, ds
    for h in range(hq):
        kh, vh = k[:, h * hkv // hq], v[:, h * hkv // hq]
        s = (q[:, h] @ kh.T * scale).masked_fill(~visible, -math.inf)
        lse[:, h] = torch.logsumexp(s, -1)
        p = torch.exp(s - lse[:, h:h + 1]).nan_to_num(0.0)
        out[:, h] = p @ vh
        ds[:, h] = (d + 8) * 2.0 ** -24 * scale * (q[:, h].abs() @ kh.abs().T).masked_fill(~visible, 0.0).amax(-1)
        weight[:, h] = p @ vh.abs()
    return out, lse, weight, ds


def check_attention(got, got_lse, ref, dtype, n_keys, v_max):
    out, lse, weight, ds = ref
    u = U[dtype]
    floor = n_keys * 2.0 ** -24 * max(v_max, 2.0) if dtype == torch.float16 else 0.0
    bound = u * out.abs() + (u + 2 * ds[..., None] + 2.0 ** -18) * weight * (1 + u) + floor + 1e-30
    err = (got.double() - out).abs()
    assert torch.isfinite(got.double()).all(), "not finite"
    assert (err <= bound).all(), f"error {(err / bound).max().item():.3f} of its bound"
    if got_lse is not None:
        empty = lse == -math.inf
        assert torch.equal(got_lse.double()[empty], lse[empty])
        e = (got_lse.double() - lse)[~empty].abs()
        b = (ds + 2.0 ** -18 * (1 + lse.abs()))[~empty]
        assert (e <= b).all(), f"lse error {(e / b).max().item():.3f} of its bound"


def norm(x, kind, w, b, eps):
    """N(x) and the size of its terms, in float64."""
    if kind == "none":
        return x, x.abs()
    mean = x.mean(-1, keepdim=True) if kind == "layer" else torch.zeros_like(x[..., :1])
    r = 1 / torch.sqrt(((x - mean) ** 2).mean(-1, keepdim=True) + eps)
    w = torch.ones_like(x) if w is None else w.double()
    b = torch.zeros_like(x) if b is None else b.double()
    return (x - mean) * r * w + b, (x.abs() + mean.abs()) * r * w.abs() + b.abs()
