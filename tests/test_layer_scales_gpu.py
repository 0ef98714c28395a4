"""Values of any size in an 8-bit cache: the softmax weights that meet their codes keep their bits."""
import math

import pytest
import torch

import attention_bounds as A

pytestmark = pytest.mark.gpu

spa = pytest.importorskip("activation_sparsification_amd")

BF16, F16 = torch.bfloat16, torch.float16
HEADS = 2048            # on one key-value head: few workgroups share its cache, so a wave walks over many tiles


def attend(dtype, fmt, page, q, k, v, scale):
    """One sequence through an 8-bit cache: out, lse and the reference on what the cache holds."""
    n, h, d = k.shape
    assert A.tiles_per_wave(spa, [n], q.shape[1], h, d) >= 6
    pages = -(-n // page)
    cache = spa.new_kv_cache(pages, page, h, d, dtype, fmt)
    spa.kv_write(k.to(dtype), v.to(dtype), torch.arange(n, dtype=torch.int32, device="cuda"), cache)
    table = torch.arange(pages, dtype=torch.int32, device="cuda")[None]
    q = q.to(dtype)
    out, lse = spa.attention_decode(q, cache, table, torch.tensor([n], dtype=torch.int32, device="cuda"), scale=scale,
                                    want_lse=True)
    held = []
    for codes, s in ((cache.k, cache.k_scale), (cache.v, cache.v_scale)):
        x = (codes.float().double() * s.double()[..., None]).transpose(1, 2).reshape(-1, h, d)
        held.append(x[:n])
    A.check(out, lse, A.reference(q, *held, scale, torch.ones((1, n), dtype=torch.bool, device="cuda")), dtype, codes=True)
    return out


def vectors(g, n, d):
    """Queries and keys whose scores are noise of about a half, and a first channel that is free."""
    q = 0.05 * torch.randn((1, HEADS, d), generator=g, device="cuda")
    k = torch.randn((n, 1, d), generator=g, device="cuda")
    q[..., 0], k[..., 0] = 1.0, 0.0
    return q, k


@pytest.mark.parametrize("fmt", ["fp8", "int8"])
@pytest.mark.parametrize("page", [16, 7])
@pytest.mark.parametrize("d", [64, 128, 96, 256])
@pytest.mark.parametrize("size,ratio", [(1.0, 3e3), (1e-2, 3e4), (1e-3, 3e4), (1e-4, 3e3), (20000.0, 3e3)])
def test_heavy_keys_without_values(fmt, page, d, size, ratio):
    # one key in sixteen tiles, in every wave's share, has a value of zero and outweighs each of the others by `ratio`:
    # what the others add, a few per cent of a small value, is the whole output
    print(f"[scales] {fmt} page {page} d {d} size {size} ratio {ratio}", flush=True)
    g = torch.Generator(device="cuda").manual_seed(d)
    n = 8200
    q, k = vectors(g, n, d)
    v = size * (1 + 0.2 * torch.randn((n, 1, d), generator=g, device="cuda"))
    pos = torch.arange(n, device="cuda")
    heavy = (pos % 32 == 5) & (pos // 32 % 16 < 4)
    k[heavy, :, 0] = 8.0
    v[heavy] = 0.0
    for dtype in (F16, BF16):
        attend(dtype, fmt, page, q, k, v, math.log(ratio) / 8)


@pytest.mark.parametrize("fmt", ["fp8", "int8"])
@pytest.mark.parametrize("page", [16, 7])
def test_sizes_that_change_along_the_sequence(fmt, page):
    # rising, falling and scattered by factors of thousands, zeros first; then the large ones hidden from the softmax
    g = torch.Generator(device="cuda").manual_seed(11)
    n, d = 6000, 128
    pos = torch.arange(n, device="cuda") / n
    sizes = {"rising": 10 ** (-4 + 7 * pos), "falling": 10 ** (3 - 7 * pos),
             "scattered": 10 ** (-3 + 4 * torch.rand(n, generator=g, device="cuda")), "zeros": (pos > 0.5).float() * 1e-3}
    for name, size in sizes.items():
        print(f"[scales] {fmt} page {page} {name}", flush=True)
        q, k = vectors(g, n, d)
        v = torch.randn((n, 1, d), generator=g, device="cuda") * size[:, None, None]
        hidden = k.clone()
        hidden[size >= 1e-2, :, 0] = -30.0
        for dtype in (F16, BF16):
            attend(dtype, fmt, page, q, k, v, 0.7)
            attend(dtype, fmt, page, q, hidden, v, 0.7)


def test_all_zero_values():
    g = torch.Generator(device="cuda").manual_seed(12)
    q, k = vectors(g, 6000, 128)
    for page in (16, 7):
        assert (attend(F16, "fp8", page, q, k, torch.zeros_like(k), 0.5) == 0).all()
