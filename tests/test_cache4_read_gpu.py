"""Reading a 4-bit cache where a wave takes several heads one after the other, and where rows are written past the caches (above
32 MiB of output): every element bit for bit, against codes times scales in 64 bits."""
import pytest
import torch

import mxfp4_ref as M

pytestmark = pytest.mark.gpu

spa = pytest.importorskip("activation_sparsification_amd")

BF16, F16, I32 = torch.bfloat16, torch.float16, torch.int32


@pytest.fixture(scope="module")
def dev():
    assert torch.cuda.is_available(), "GPU tests need a device"
    return torch.device("cuda:0")


def filled(dev, g, dtype, n_pages, page, h, d):
    """A cache of every code, scales whose products are normal numbers of the type, some groups of zeros and of NaN; its values."""
    cache = spa.new_kv_cache(n_pages, page, h, d, dtype, "mxfp4", dev)
    lo, hi = (27, 253) if dtype == BF16 else (127 - 12, 127 + 14)
    held = []
    for pages, scales in ((cache.k, cache.k_scale), (cache.v, cache.v_scale)):
        pages.copy_(torch.randint(0, 256, pages.shape, generator=g, device=dev).to(torch.uint8))
        scales.copy_(torch.randint(lo, hi, scales.shape, generator=g, device=dev).to(torch.uint8))
        odd = torch.rand(scales.shape, generator=g, device=dev)
        scales[odd < 0.01] = 255
        scales[odd > 0.99] = 0
        none = ((odd < 0.01) | (odd > 0.99)).transpose(-1, -2).repeat_interleave(16, dim=-1)[..., :d // 2]
        pages[none] = 0                                          # as such groups are stored
        held.append(M.values(pages, scales))
    return cache, held


@pytest.mark.parametrize("lens,h,d,page,dtype", [
    # below 32 MiB: two rounds of heads to a wave, a tail of one head, shares of 12 and 10 heads, five rounds
    ([2500, 1, 0, 1700, 17, 900], 8, 64, 16, BF16),
    ([5000], 5, 128, 32, F16),
    ([1500, 33, 1400], 22, 40, 7, BF16),
    ([2100, 2100, 15], 20, 64, 16, F16),
    ([4700], 6, 8, 24, BF16),
    # above 32 MiB, rows written past the caches: one to five rounds, shares of 12 heads and 4
    ([6000, 1, 0, 3500, 17, 900], 8, 128, 16, BF16),
    ([9001, 12000, 63, 6000], 5, 64, 32, F16),
    ([3300, 7, 3300], 20, 64, 16, BF16),
    ([4001, 900, 1], 9, 256, 16, F16),
    ([2800, 2801], 16, 96, 7, BF16),
    ([70001], 2, 64, 64, BF16),
    ([1100, 900, 31], 40, 128, 16, F16),
])
def test_read_of_many_rows(dev, lens, h, d, page, dtype):
    print(f"[read] {dtype} {lens} heads {h}x{d} page {page}", flush=True)
    g = torch.Generator(device=dev).manual_seed(h * d + page)
    need = [-(-x // page) for x in lens]
    n_pages = sum(need) + 3
    cache, held = filled(dev, g, dtype, n_pages, page, h, d)
    perm = torch.randperm(n_pages, generator=g, device=dev).to(I32)
    table = torch.full((len(lens), max(need)), 2 ** 31 - 1, dtype=I32, device=dev)
    at = 0
    for s, x in enumerate(need):
        table[s, :x] = perm[at:at + x]
        at += x
    table[0, need[0] // 2], table[0, need[0] - 1] = -1, n_pages  # absent pages
    cu = torch.tensor([0] + lens).cumsum(0).to(I32).to(dev)
    total = sum(lens) + 5
    outs = [torch.full((total, h, d), 7.0, dtype=dtype, device=dev) for _ in range(2)]
    spa.kv_read(cache, table, cu, total, k_out=outs[0], v_out=outs[1])
    at = 0
    for s, x in enumerate(lens):
        pos = torch.arange(x, device=dev)
        pg = table[s, pos // page].long()
        there = (pg >= 0) & (pg < n_pages)
        for got, y in zip(outs, held):
            want = torch.where(there[:, None, None], y[pg.clamp(0, n_pages - 1), :, pos % page], torch.zeros((), dtype=torch.float64, device=dev))
            assert torch.equal(got[at:at + x].isnan(), want.isnan())
            assert torch.equal(got[at:at + x].nan_to_num(), want.to(dtype).nan_to_num())
        at += x
    assert all((got[at:] == 7).all() for got in outs)            # rows behind the last sequence


def test_streamed_rows_are_there_for_the_next_call(dev):
    # written past the caches, read by the attention that follows at once; every replay of a capture as well
    g = torch.Generator(device=dev).manual_seed(5)
    h, d, n = 8, 128, 9000
    cache, _ = filled(dev, g, BF16, -(-n // 16), 16, h, d)
    for s in (cache.k_scale, cache.v_scale):
        s.copy_(torch.randint(122, 128, s.shape, generator=g, device=dev).to(torch.uint8))
    table = torch.randperm(-(-n // 16), generator=g, device=dev).to(I32)[None]
    cu_q, cu = torch.tensor([0, 3], dtype=I32, device=dev), torch.tensor([0, n], dtype=I32, device=dev)
    q = torch.randn((3, h, d), generator=g, device=dev).to(BF16)
    k, v = (torch.empty((n, h, d), dtype=BF16, device=dev) for _ in range(2))
    out = torch.empty_like(q)

    def step():
        spa.kv_read(cache, table, cu, n, k_out=k, v_out=v)
        spa.attention_prefill(q, k, v, cu_q, cu, out=out)

    step()
    torch.cuda.synchronize()
    want = out.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for _ in range(3):
        for x in (k, v, out):
            x.fill_(9.0)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)
