"""A 64-bit attention of one sequence and two error bounds that tell a misread tile from rounding.

``reference`` returns the outputs with what the bounds need of them.  ``check`` holds every output to the sum of the
roundings that the library's definition allows, and all outputs together to their root sum square:

* each output is rounded once: u |o|, no less than the last place of a subnormal;
* each softmax weight carries the 16-bit rounding u before it meets its value, the float32 error of its score,
  2 ds with ds = (d + 8) 2^-24 scale sum |q k|, and 2^-18 for the exponential; these errors belong to the key, so over
  the keys they add up like independent numbers: by the root of sum (p v)^2, where sum p |v| bounds one output alone;
* the scale's own rounding shifts all scores of a row by one factor: (1 + max |s|) 2^-22 of sum p |v|;
* a float16 weight below 2^-14 loses up to 2^-25 of the largest weight, which is S = sum exp(s - max s) of the row's
  sum: 2^-25 |v| / S for each key.  Codes of an 8-bit cache meet weights that carry the value's scale, brought to 2^14 at
  the largest: 2^-38 max |v| / S for each key.

A root sum square of errors of up to their bounds is reached only when all of them are at their ends; 1.5 times the
root covers rows of one or two keys, where the number of independent errors is small.
"""
import math

import torch

U = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
TINY = {torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25}     # half the last place of a subnormal


def reference(q, k, v, scale, visible):
    """One sequence: q [lq, hq, d], k and v [lk, hkv, d], visible [lq, lk] bool; everything finite that is visible."""
    q, k, v = q.double(), k.double(), v.double()
    lq, hq, d = q.shape
    lk, hkv = k.shape[:2]
    r = {"out": torch.zeros_like(q), "lse": torch.full((lq, hq), -math.inf, dtype=torch.float64, device=q.device)}
    for name in ("pv", "pv2", "v", "v2"):
        r[name] = torch.zeros_like(q)
    for name in ("ds", "smax", "top"):
        r[name] = torch.zeros_like(r["lse"])
    r["top"] += 1.0
    r["vmax"] = float(v.abs().max()) if lk else 0.0
    r["keys"] = visible.sum(-1).double()[:, None, None]
    if lk == 0 or lq == 0:
        return r
    seen = visible.double()
    for h in range(hkv):
        heads = slice(h * hq // hkv, (h + 1) * hq // hkv)
        qh, kh, vh = q[:, heads].transpose(0, 1), k[:, h], v[:, h]                  # [g, lq, d], [lk, d]
        s = (qh.reshape(-1, d) @ kh.T.contiguous() * scale).view(-1, lq, lk)
        size = (qh.abs().reshape(-1, d) @ kh.T.abs().contiguous() * scale).view(-1, lq, lk)
        size = size.masked_fill(~visible, 0.0).amax(-1)
        s = s.masked_fill(~visible, -math.inf)
        m = s.amax(-1, keepdim=True)
        base = torch.where(m == -math.inf, torch.zeros_like(m), m)
        e = torch.exp(s - base)
        total = e.sum(-1, keepdim=True)
        p = e / torch.where(total > 0, total, torch.ones_like(total))
        flat = p.reshape(-1, lk)

        def put(name, x):
            r[name][:, heads] = x.view(-1, lq, d).transpose(0, 1)

        put("out", flat @ vh)
        put("pv", flat @ vh.abs())
        put("pv2", flat.square() @ vh.square())
        r["v"][:, heads] = (seen @ vh.abs())[:, None]
        r["v2"][:, heads] = (seen @ vh.square())[:, None]
        r["lse"][:, heads] = (base + total.log()).squeeze(-1).T
        r["top"][:, heads] = total.squeeze(-1).clamp(min=1.0).T
        r["ds"][:, heads] = ((d + 8) * 2.0 ** -24 * size).T
        r["smax"][:, heads] = s.masked_fill(~visible, 0.0).abs().amax(-1).T
    return r


def check(got, got_lse, r, dtype, codes=False):
    """Raises AssertionError unless outputs (and log-sum-exps, or None) lie within the bounds.  codes: an 8-bit cache."""
    u, out = U[dtype], r["out"]
    if out.numel() == 0:
        return
    assert torch.isfinite(got.double()).all(), "not finite"
    err = (got.double() - out).abs()
    own = torch.maximum(u * out.abs(), torch.full_like(out, TINY[dtype]))
    weight = u + 2 * r["ds"][..., None] + 2.0 ** -18
    shift = (1 + r["smax"])[..., None] * 2.0 ** -22 * r["pv"]
    if dtype != torch.float16:
        low = low2 = torch.zeros_like(out)
    elif codes:
        low = 2.0 ** -38 * r["vmax"] * r["keys"] / r["top"][..., None]
        low2 = low.square() / r["keys"].clamp(min=1.0)
    else:
        low = 2.0 ** -25 * r["v"] / r["top"][..., None]
        low2 = 2.0 ** -50 * r["v2"] / r["top"][..., None].square()
    bound = (own + weight * r["pv"] + shift + low) * (1 + u) + 1e-300
    assert (err <= bound).all(), f"error {(err / bound).max().item():.3f} of its bound"
    rss = 1.5 * (own.square() + weight.square() * r["pv2"] + shift.square() + low2).sum().sqrt() + 1e-300
    assert err.square().sum().sqrt() <= rss, f"error {(err.square().sum().sqrt() / rss).item():.3f} of its bound over all"
    if got_lse is not None:
        lse = r["lse"]
        empty = lse == -math.inf
        assert torch.equal(got_lse.double()[empty], lse[empty])
        e = (got_lse.double() - lse)[~empty].abs()
        b = (r["ds"] + 2.0 ** -18 * (1 + lse.abs()))[~empty]
        assert (e <= b).all(), f"lse error {(e / b).max().item():.3f} of its bound"


def as_computed(q, k, v, scale, visible, dtype):
    """What a correct kernel gives: weights and outputs rounded to ``dtype``, the rest exact.  Shapes as ``reference``."""
    q, k, v = q.double(), k.double(), v.double()
    hq, hkv, d = q.shape[1], k.shape[1], q.shape[2]
    out = torch.zeros_like(q)
    for h in range(hkv):
        heads = slice(h * hq // hkv, (h + 1) * hq // hkv)
        s = torch.einsum("igd,jd->gij", q[:, heads], k[:, h]) * scale
        s = s.masked_fill(~visible, -math.inf)
        e = torch.exp(s - s.amax(-1, keepdim=True).clamp(min=-1e300))
        w = e.to(dtype).double()
        out[:, heads] = torch.einsum("gij,jd->igd", w, v[:, h]) / e.sum(-1).T[..., None].clamp(min=1e-300)
    return out.to(dtype)


def tiles_per_wave(spa, lens, hq, hkv, d):
    """Tiles of 32 positions that a wave of decode attention walks one after the other: the tiles of all sequences are
    shared by the workgroups of a head (their number is in the workspace's size), a workgroup's by its four waves."""
    up = lambda x: -(-x // 256) * 256
    size = spa.lib().spa_attention_decode_workspace_bytes(len(lens), hq, hkv, d)
    groups = [g for g in range(1, 1025) if up(2 * g * hq * d * 4) + up(2 * g * hq * 8) + up(len(lens) * 8) == size]
    assert len(groups) == 1
    tiles = sum(max(-(-x // 32), 1) for x in lens)
    return -(-max(-(-tiles // groups[0]), 4) // 4)
