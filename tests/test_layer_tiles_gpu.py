"""Decode attention where a wave walks over many tiles: keys in flight across tiles, page numbers refilled, maxima that rise
late, absent pages in the middle, on every format, type and kind of page."""
import pytest
import torch

import attention_bounds as A

pytestmark = pytest.mark.gpu

spa = pytest.importorskip("activation_sparsification_amd")

BF16, F16 = torch.bfloat16, torch.float16
NAMES = {BF16: "bf16", F16: "f16"}


def walk(dtype, fmt, hq, hkv, d, page, lens, tiles, rising=0.0, absent=(), seed=0):
    """Sequences on shuffled pages against the reference.  tiles: how many a wave walks over, at the least and at the most.
    rising: the scores grow by this much from the first position to the last.  absent: (sequence, column) of the table."""
    n_tiles = A.tiles_per_wave(spa, lens, hq, hkv, d)
    print(f"[tiles] {NAMES[dtype]} {fmt} heads {hq}/{hkv}x{d} page {page} lens {lens} tiles of a wave {n_tiles}", flush=True)
    assert tiles[0] <= n_tiles <= tiles[1]
    g = torch.Generator(device="cuda").manual_seed(seed + d + page)
    need = [-(-x // page) for x in lens]
    n_pages = sum(need) + 2
    perm = torch.randperm(n_pages, generator=g, device="cuda").to(torch.int32)
    table = torch.full((len(lens), max(need)), -1, dtype=torch.int32, device="cuda")
    cache = spa.new_kv_cache(n_pages, page, hkv, d, dtype, fmt)
    q = torch.randn((len(lens), hq, d), generator=g, device="cuda")
    q[..., 0] = 2.0
    at = 0
    for s, x in enumerate(lens):
        table[s, :need[s]] = perm[at:at + need[s]]
        at += need[s]
        if x:
            pos = torch.arange(x, device="cuda")
            k, v = (torch.randn((x, hkv, d), generator=g, device="cuda") for _ in range(2))
            k[..., 0] = (rising * d ** 0.5 / 2 * (pos / x - 0.5))[:, None]
            slots = (table[s, pos // page].long() * page + pos % page).to(torch.int32)
            spa.kv_write(k.to(dtype), v.to(dtype), slots, cache)
    full = table.clone()
    for s, column in absent:
        table[s, column] = -1 if column % 2 else n_pages
    q = q.to(dtype)
    out, lse = spa.attention_decode(q, cache, table, torch.tensor(lens, dtype=torch.int32, device="cuda"), want_lse=True)
    for s, x in enumerate(lens):
        pos = torch.arange(x, device="cuda")
        gone = torch.zeros(x, dtype=torch.bool, device="cuda")
        for t, column in absent:
            if t == s:
                gone |= pos // page == column
        pos = pos[~gone]
        slot = full[s, pos // page].long(), pos % page
        held = []
        for codes, scale in ((cache.k, cache.k_scale), (cache.v, cache.v_scale)):
            y = codes.view(torch.int8)[slot[0], :, slot[1]].view(codes.dtype).double() if codes.element_size() == 1 else \
                codes[slot[0], :, slot[1]].double()
            held.append(y if scale is None else y * scale[slot[0], :, slot[1]].double()[..., None])
        r = A.reference(q[s:s + 1], *held, d ** -0.5, torch.ones((1, len(pos)), dtype=torch.bool, device="cuda"))
        A.check(out[s:s + 1], lse[s:s + 1], r, dtype, codes=fmt != "native")


FORMATS = ["native", "fp8", "int8"]


# 1024 query heads on two key-value heads are 32 tiles of heads each: 8 workgroups share a head's cache at a head_dim of up
# to 128, 12 to 64, 4 to 256
@pytest.mark.parametrize("fmt", ["fp8", "int8"])
@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("d", [8, 24, 40, 72, 104, 136, 200, 248])
def test_rows_that_start_on_8_bytes(fmt, dtype, d):
    walk(dtype, fmt, 1024, 2, d, 16, [2500, 3001], (4, 12))


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("d", [64, 128, 256, 40, 96, 200])
@pytest.mark.parametrize("page", [16, 48, 7, 8])
def test_tiles_of_a_wave(fmt, dtype, d, page):
    walk(dtype, fmt, 1024, 2, d, page, [6001, 3, 4100, 0, 777], (6, 24))
    walk(dtype, fmt, 1024, 2, d, page, [6001, 3, 4100, 0, 777], (6, 24), rising=12.0, seed=1)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("d,n", [(64, 60000), (128, 40000), (256, 20000), (96, 40000)])
@pytest.mark.parametrize("page", [16, 7])
def test_more_tiles_than_page_numbers_held(fmt, dtype, d, n, page):
    # a wave holds the page numbers of 32 tiles and reads the next ones on its way
    walk(dtype, fmt, 1024, 2, d, page, [n, 5, n // 3 + 1], (33, 64), rising=6.0)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("page", [16, 32, 7])
def test_absent_pages_on_the_way(fmt, page):
    last = 5000 // page
    gone = [(0, c) for c in (0, 1, 17, 18, 19, 20, 100, last - 1)] + [(1, c) for c in range(40)] + [(2, 3)]
    walk(BF16, fmt, 1024, 2, 128, page, [5000, 3000, 6000], (10, 24), absent=gone, rising=8.0)
    walk(F16, fmt, 1024, 2, 72, page, [5000, 3000, 6000], (10, 24), absent=gone)


def test_many_key_value_heads():
    # 32 key-value heads leave 16 workgroups to each
    walk(BF16, "fp8", 32, 32, 128, 16, [30000, 9000], (17, 32), rising=6.0)
    walk(F16, "int8", 64, 32, 64, 16, [20000, 17], (6, 16))
