"""The 4-bit cache format in 64 bits: e2m1 codes with one power-of-two scale for every 32 elements of a vector.

The largest magnitude a of the 32 sets the exponent: the least e with a <= 7 * 2^e, at most 13 (float16) or 125
(bfloat16).  Codes are the nearest of 0, 0.5, 1, 1.5, 2, 3, 4, 6 to |x| / 2^e (ties to the even code) with the sign of x.
"""
import torch

GRID = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
TOP = {torch.float16: 13, torch.bfloat16: 125}


def quantise(x, dtype):
    """Codes (0..15) [..., d] and exponent bytes [..., ceil(d / 32)] of float vectors of ``dtype``'s range."""
    x = x.double()
    grid = torch.tensor(GRID, dtype=torch.float64, device=x.device)
    codes, scales = [], []
    for i in range(0, x.shape[-1], 32):
        g = x[..., i:i + 32]
        a = g.abs().amax(-1, keepdim=True)
        bad = ~torch.isfinite(g).all(-1, keepdim=True)
        live = ~bad & (a >= 2.0 ** -100)
        safe = torch.where(live, a, torch.ones_like(a))
        e = torch.full_like(safe, -110.0)
        for up in range(-110, TOP[dtype] + 1):                  # by trial: no logarithm
            e = torch.where(safe > 7 * 2.0 ** (up - 1), torch.full_like(e, float(up)), e)
        y = (torch.where(live, g, torch.zeros_like(g)) / torch.exp2(e)).abs()
        cost = (y[..., None] - grid).abs()
        best = cost.amin(-1, keepdim=True)
        hit = cost == best                                      # two where y is half way: the even one
        code = torch.where(hit & (torch.arange(8, device=x.device) % 2 == 0), 0, torch.where(hit, 1, 2)).argmin(-1)
        code = code + 8 * torch.signbit(g)
        codes.append(torch.where(live, code, torch.zeros_like(code)))
        scales.append(torch.where(bad, torch.full_like(e, 255.0), torch.where(live, e + 127, torch.zeros_like(e))))
    return torch.cat(codes, dim=-1), torch.cat(scales, dim=-1).long()


def pack(codes):
    """Codes [..., d] as bytes [..., d / 2]."""
    return (codes[..., 0::2] + 16 * codes[..., 1::2]).to(torch.uint8)


def values(pages, scales):
    """Pages [n, h, page, d / 2] and scales [n, h, groups, page] as float64 [n, h, page, d]."""
    nibbles = torch.stack([pages & 15, pages >> 4], dim=-1).flatten(-2).long()
    grid = torch.tensor(GRID + tuple(-x for x in GRID), dtype=torch.float64, device=pages.device)
    s = scales.transpose(-1, -2).double()
    s = torch.where(s == 255, torch.full_like(s, float("nan")), torch.exp2(s - 127))
    return grid[nibbles] * s.repeat_interleave(32, dim=-1)[..., :nibbles.shape[-1]]


def fill(cache, g, dtype, gain=1.0):
    """Random vectors in every place of a cache, quantised by the reference; the values that it stands for."""
    n, h, page, half = cache.k.shape
    held = []
    for pages, scales in ((cache.k, cache.k_scale), (cache.v, cache.v_scale)):
        x = (torch.randn((n, h, page, 2 * half), generator=g, device=pages.device) * gain).to(dtype)
        c, s = quantise(x, dtype)
        pages.copy_(pack(c))
        scales.copy_(s.transpose(-1, -2).to(torch.uint8))
        held.append(values(pages, scales))
    return held
