"""Softmax weights of decode attention over the 4-bit cache keep 16 bits, for both types of vectors.

An output is off by u |y| for its own rounding and, relative to sum p |v| of its keys, by
* 2^-16 for its weights, the sum of two bfloat16 numbers, each rounded by at most 2^-8 of what it holds;
* 2^-16 for the products' sums: fewer than 128 additions in a row (32 positions and both parts of a tile, 16 tiles of a wave, the
  joins), each off by at most 2^-23 whichever way the matrix unit rounds;
* 2^-18 for the exponential and 2 ds for the scores: (d + 8) 2^-24 scale sum |q k| and the holding of query elements
  to 2^-19 of the largest of their 32;
* (1 + max |s|) 2^-22 for the rounding of the scale, one factor of all scores of a row.
Weights of 8 bits, as bfloat16 holds one, are off by 2^-8 and leave these bounds where values cancel.
"""
import pytest
import torch

import attention_bounds as A
import mxfp4_ref as M

pytestmark = pytest.mark.gpu

spa = pytest.importorskip("activation_sparsification_amd")

BF16, F16, I32 = torch.bfloat16, torch.float16, torch.int32
FIXED = 2.0 ** -16 + 2.0 ** -16 + 2.0 ** -18


@pytest.fixture(scope="module")
def dev():
    assert torch.cuda.is_available(), "GPU tests need a device"
    return torch.device("cuda:0")


def check(got, y, pv, weight, dtype):
    u = A.U[dtype]
    own = torch.maximum(u * y.abs(), torch.full_like(y, A.TINY[dtype]))
    err = (got.double() - y).abs()
    bound = (own + weight * pv) * (1 + u)
    assert (err <= bound).all(), f"error {(err / bound).max().item():.3f} of its bound"


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("page", [16, 5])
@pytest.mark.parametrize("hq,d", [(1, 64), (3, 128), (6, 96), (16, 256)])
def test_two_positions_that_cancel(dev, dtype, page, hq, d):
    # values 6 and -6 with weights 1 and exp(s) before the division: y = 6 (1 - exp(s)) / (1 + exp(s))
    n = 64
    cache = spa.new_kv_cache(n, page, 1, d, dtype, "mxfp4", dev)
    cache.k_scale.fill_(127)
    cache.v_scale.fill_(127)
    cache.k[:, :, 1, 0] = 2                                     # position 1: the first element is 1
    cache.v[:, :, 0], cache.v[:, :, 1] = 0x77, 0xFF
    s = -torch.arange(1, n + 1, device=dev) / 128.0             # exact in both types
    q = torch.zeros((n, hq, d), dtype=dtype, device=dev)
    q[:, :, 0] = s[:, None].to(dtype)
    table = torch.arange(n, dtype=I32, device=dev)[:, None]
    got, _ = spa.attention_decode(q, cache, table, torch.full((n,), 2, dtype=I32, device=dev), scale=1.0)
    e = s.double().exp()
    y = (6 * (1 - e) / (1 + e))[:, None, None].expand(n, hq, d)
    shift = (1 + s.double().abs()) * 2.0 ** -22
    # one product makes the score: 9 * 2^-24 |s| and the holding of the query, 2^-19 |s|
    ds = (9 * 2.0 ** -24 + 2.0 ** -19) * s.double().abs()
    check(got, y, torch.full_like(y, 6.0), (FIXED + shift + 2 * ds)[:, None, None], dtype)


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("hq,hkv,d,page", [(8, 2, 128, 16), (4, 4, 64, 32), (20, 1, 64, 16), (6, 3, 96, 7), (2, 1, 256, 16), (10, 2, 200, 16)])
def test_random_values(dev, dtype, hq, hkv, d, page):
    g = torch.Generator(device=dev).manual_seed(d + hq)
    lens = [1000, 1, 2, 33, 517]
    need = [-(-x // page) for x in lens]
    cache = spa.new_kv_cache(sum(need), page, hkv, d, dtype, "mxfp4", dev)
    held = M.fill(cache, g, dtype)
    perm = torch.randperm(sum(need), generator=g, device=dev).to(I32)
    q = torch.randn((len(lens), hq, d), generator=g, device=dev).to(dtype)
    scale = d ** -0.5
    for width in (max(need), -(-4000 // page)):                 # sequences whole, and cut
        table = torch.full((len(lens), width), -1, dtype=I32, device=dev)
        at = 0
        for i, x in enumerate(need):
            table[i, :x] = perm[at:at + x]
            at += x
        got, _ = spa.attention_decode(q, cache, table, torch.tensor(lens, dtype=I32, device=dev), scale=scale)
        for i, x in enumerate(lens):
            pos = torch.arange(x, device=dev)
            k, v = (y[table[i, pos // page].long(), :, pos % page] for y in held)
            r = A.reference(q[i:i + 1], k, v, scale, torch.ones((1, x), dtype=torch.bool, device=dev))
            hold = sum(q[i, :, b:b + 32].double().abs().amax(-1) * k[..., b:b + 32].abs().sum(-1).amax(0).repeat_interleave(hq // hkv)
                       for b in range(0, d, 32))
            ds = r["ds"] + 2.0 ** -19 * scale * hold
            weight = FIXED + 2 * ds + (1 + r["smax"]) * 2.0 ** -22
            check(got[i:i + 1], r["out"], r["pv"], weight[..., None], dtype)
