"""The 4-bit cache on the GPU: codes and scales bit for bit, reading back, and decode attention within bounds that are summed
from its roundings (tests/attention_bounds.py).

Beside those bounds a query element is held to 2^-19 of the largest of its 32, so a score is off by up to 2^-19 scale sum
over the blocks of max |q| sum |k|; QUERY_ERROR below.  The weights of a float16 call keep 16 bits, finer than the bounds ask.
"""
import math
import random

import pytest
import torch

import attention_bounds as A
import mxfp4_ref as M

pytestmark = pytest.mark.gpu

spa = pytest.importorskip("activation_sparsification_amd")

BF16, F16, I32 = torch.bfloat16, torch.float16, torch.int32
NAMES = {BF16: "bf16", F16: "f16"}


@pytest.fixture(scope="module")
def dev():
    assert torch.cuda.is_available(), "GPU tests need a device"
    return torch.device("cuda:0")


def gen(dev, seed):
    return torch.Generator(device=dev).manual_seed(seed)


def table_for(dev, g, lens, page, n_pages):
    """Shuffled pages; unused entries of the table are far out of range."""
    need = [-(-x // page) for x in lens]
    perm = torch.randperm(n_pages, generator=g, device=dev).to(I32)
    table = torch.full((len(lens), max(need + [1])), 2 ** 31 - 1, dtype=I32, device=dev)
    at = 0
    for s, x in enumerate(need):
        table[s, :x] = perm[at:at + x]
        at += x
    return table


# ---------------------------------------------------------------------------------------------------------------
# writing and reading
# ---------------------------------------------------------------------------------------------------------------
def special(dtype, d, dev):
    """Vectors whose groups sit on the format's edges."""
    big = torch.finfo(dtype).max
    rows = [torch.zeros(d), torch.full((d,), 1.0), torch.full((d,), -7.0), torch.full((d,), 7.0 + 2 ** -4), torch.full((d,), big),
            torch.full((d,), -0.0)]
    grid = torch.tensor([6.0, 0.25, -0.25, 0.75, 1.25, -1.75, 2.5, 3.5, 5.0, 7.0, -0.2, 0.3, 0.0, -0.0, 4.9, 5.1])
    rows += [grid.repeat(16)[:d], grid.repeat(16)[:d] * 2.0 ** -20, grid.flip(0).repeat(16)[:d] * 3]
    if dtype == BF16:
        rows += [torch.full((d,), 2.0 ** -101), torch.full((d,), 2.0 ** -100), grid.repeat(16)[:d] * 2.0 ** -99,
                 grid.repeat(16)[:d] * 2.0 ** 124]
    else:
        rows += [torch.full((d,), 2.0 ** -24), torch.full((d,), 57344.0), torch.full((d,), 57376.0)]
    bad = torch.randn(d)
    bad[d // 2] = math.nan
    worse = torch.randn(d)
    worse[0] = -math.inf
    return torch.stack(rows + [bad, worse]).to(dtype).to(dev)


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("t,h,d,page", [(1, 1, 8, 1), (33, 3, 40, 7), (64, 8, 128, 16), (50, 2, 256, 100), (41, 4, 64, 32),
                                        (300, 5, 96, 16), (30, 1, 32, 5)])
def test_write(dev, dtype, t, h, d, page):
    print(f"[write] {NAMES[dtype]} t {t} heads {h}x{d} page {page}", flush=True)
    g = gen(dev, t + d)
    n_pages = -(-t // page) + 3
    cache = spa.new_kv_cache(n_pages, page, h, d, dtype, "mxfp4", dev)
    assert (cache.n_pages, cache.page_size, cache.n_heads, cache.head_dim) == (n_pages, page, h, d)
    x = (torch.randn((t, 2 * h + 1, d), generator=g, device=dev) * 3).to(dtype)
    edge = special(dtype, d, dev)[:t]
    x[:len(edge), 0], x[:len(edge), h] = edge, edge
    k, v = x[:, :h], x[:, h:2 * h]
    slots = torch.randperm(n_pages * page, generator=g, device=dev)[:t].to(I32)
    skip = torch.rand(t, generator=g, device=dev) < 0.1
    slots[skip] = -1
    if t > 30:
        slots[28], slots[29] = n_pages * page, 2 ** 31 - 1      # past the cache: skipped as well
        skip[28:30] = True
    marked = [cache.k, cache.v, cache.k_scale, cache.v_scale]
    for b in marked:
        b.fill_(0x35)
    want = [b.clone() for b in marked]
    spa.kv_write(k, v, slots, cache)
    live = (~skip).nonzero().squeeze(-1)
    pg, off = slots[live].long() // page, slots[live].long() % page
    for i, rows in enumerate((k[live], v[live])):
        codes, scales = M.quantise(rows, dtype)
        want[i][pg, :, off] = M.pack(codes)
        want[2 + i][pg, :, :, off] = scales.to(torch.uint8)
    for got, w, name in zip(marked, want, ("k", "v", "k_scale", "v_scale")):
        assert torch.equal(got, w), name


def test_no_value_leaves_the_type(dev):
    # the largest finite numbers and what is near them read back finite, within half a step of the scale's top codes
    for dtype in (BF16, F16):
        x = special(dtype, 64, dev)
        x = x[torch.isfinite(x).all(-1)][:, None]
        cache = spa.new_kv_cache(2, 16, 1, 64, dtype, "mxfp4", dev)
        spa.kv_write(x, x, torch.arange(len(x), dtype=I32, device=dev), cache)
        got, _ = spa.kv_read(cache, torch.tensor([[0, 1]], dtype=I32, device=dev), torch.tensor([0, len(x)], dtype=I32, device=dev),
                             len(x), dtype=dtype)
        assert torch.isfinite(got).all()
        a = x.double().abs().amax(-1, keepdim=True)
        assert ((got.double() - x.double()).abs() <= a * 2 / 7 + 2.0 ** -100).all()


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("lens,h,d,page", [([1], 1, 8, 1), ([0, 5, 0, 33], 3, 40, 7), ([100, 1, 16, 17], 8, 128, 16), ([300], 2, 256, 64),
                                           ([63, 64, 65], 4, 64, 32), ([31, 200], 2, 96, 16)])
def test_read(dev, dtype, lens, h, d, page):
    print(f"[read] {NAMES[dtype]} {lens} heads {h}x{d} page {page}", flush=True)
    g = gen(dev, d)
    n_pages = sum(-(-x // page) for x in lens) + 4
    cache = spa.new_kv_cache(n_pages, page, h, d, dtype, "mxfp4", dev)
    held = M.fill(cache, g, dtype)
    cache.k_scale[0, 0, 0, 0] = 255
    held[0] = M.values(cache.k, cache.k_scale)
    table = table_for(dev, g, lens, page, n_pages)
    cu = torch.tensor([0] + lens).cumsum(0).to(I32).to(dev)
    total = sum(lens) + 5
    k_out, v_out = (torch.full((total, h, d), 7.0, dtype=dtype, device=dev) for _ in range(2))
    spa.kv_read(cache, table, cu, total, k_out=k_out, v_out=v_out)
    at = 0
    for s, x in enumerate(lens):
        pos = torch.arange(x, device=dev)
        pg = table[s, pos // page].long()
        for got, y in ((k_out, held[0]), (v_out, held[1])):
            want = y[pg, :, pos % page].to(dtype)
            assert torch.equal(got[at:at + x].nan_to_num(nan=-99.0), want.nan_to_num(nan=-99.0))
        at += x
    assert (k_out[at:] == 7).all() and (v_out[at:] == 7).all()          # rows behind the last sequence


def test_read_absent_pages_are_zero(dev):
    g = gen(dev, 1)
    cache = spa.new_kv_cache(6, 8, 2, 64, BF16, "mxfp4", dev)
    held = M.fill(cache, g, BF16)
    table = torch.tensor([[2, -1, 5], [6, 0, 1]], dtype=I32, device=dev)
    cu = torch.tensor([0, 40, 60], dtype=I32, device=dev)               # the first sequence is longer than its table
    k, v = spa.kv_read(cache, table, cu, 60, dtype=BF16)
    for got, y in ((k, held[0]), (v, held[1])):
        want = torch.zeros((60, 2, 64), dtype=torch.float64, device=dev)
        for s, (a, b) in enumerate(((0, 40), (40, 60))):
            for i in range(b - a):
                pg = int(table[s, i // 8]) if i // 8 < 3 else -1
                if 0 <= pg < 6:
                    want[a + i] = y[pg, :, i % 8]
        assert torch.equal(got.double(), want)


# ---------------------------------------------------------------------------------------------------------------
# attention
# ---------------------------------------------------------------------------------------------------------------
def query_error(q, k, scale):
    """What holding query elements to 2^-19 of the largest of their 32 can change in a score: q [1, hq, d], k [lk, hkv, d]."""
    hq, hkv = q.shape[1], k.shape[1]
    most = torch.zeros((1, hq), dtype=torch.float64, device=q.device)
    for i in range(0, q.shape[-1], 32):
        a = q[..., i:i + 32].double().abs().amax(-1)
        size = k[..., i:i + 32].abs().sum(-1).amax(0)
        most += a * size.repeat_interleave(hq // hkv)
    return 2.0 ** -19 * scale * most


def decode_check(dev, dtype, hq, hkv, d, page, lens, seed=0, scale=None, gain=1.0, absent=(), quiet=False, outlier=1.0, room=0):
    if not quiet:
        print(f"[decode] {NAMES[dtype]} heads {hq}/{hkv}x{d} page {page} lens {lens[:8]}", flush=True)
    g = gen(dev, seed + d + page)
    n_pages = sum(-(-x // page) for x in lens) + 2
    cache = spa.new_kv_cache(n_pages, page, hkv, d, dtype, "mxfp4", dev)
    held = M.fill(cache, g, dtype, gain)
    table = table_for(dev, g, lens, page, n_pages)
    wider = -(-room // page) - table.shape[1]
    if wider > 0:                       # a table of `room` positions to a sequence, as for sequences that go on
        table = torch.nn.functional.pad(table, (0, wider), value=2 ** 31 - 1).contiguous()
    full = table.clone()
    for s, column in absent:
        table[s, column] = -1 if column % 2 else n_pages
    q = torch.randn((len(lens), hq, d), generator=g, device=dev)
    q[..., d // 3] *= outlier
    q = q.to(dtype)
    out, lse = spa.attention_decode(q, cache, table, torch.tensor(lens, dtype=I32, device=dev), scale=scale, want_lse=True)
    sc = d ** -0.5 if scale is None else scale
    for s, x in enumerate(lens):
        pos = torch.arange(x, device=dev)
        for t, column in absent:
            if t == s:
                pos = pos[pos // page != column]
        k, v = (y[full[s, pos // page].long(), :, pos % page] for y in held)
        r = A.reference(q[s:s + 1], k, v, sc, torch.ones((1, len(pos)), dtype=torch.bool, device=dev))
        if len(pos):
            r["ds"] = r["ds"] + query_error(q[s:s + 1], k, sc)
        A.check(out[s:s + 1], lse[s:s + 1], r, dtype, codes=True)
    return out, lse


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("hq,hkv,d", [(1, 1, 8), (4, 4, 64), (8, 2, 128), (6, 3, 96), (2, 1, 256), (4, 2, 40), (2, 2, 160), (40, 1, 128),
                                      (20, 1, 64), (3, 1, 32), (5, 1, 200)])
def test_decode_heads(dev, dtype, hq, hkv, d):
    for page in (16, 7):
        decode_check(dev, dtype, hq, hkv, d, page, [1, 0, 33, 70, 200], seed=hq)


@pytest.mark.parametrize("page", [1, 5, 16, 48, 100, 256])
def test_decode_pages(dev, page):
    for dtype, d in ((BF16, 128), (F16, 64)):
        decode_check(dev, dtype, 4, 2, d, page, [1, 15, 16, 17, 31, 32, 33, 127, 128, 129, 500, 0])


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("page", [16, 24])
def test_decode_long(dev, dtype, page):
    # many tiles to a wave, sequences cut between workgroups and joined
    decode_check(dev, dtype, 4, 1, 128, page, [70001, 3, 9000])
    decode_check(dev, dtype, 2, 2, 64, page, [30000, 30001])
    decode_check(dev, dtype, 2, 1, 256, page, [20000])


@pytest.mark.parametrize("n,longest,d,hkv", [(3, 9000, 128, 8), (40, 1500, 128, 8), (130, 700, 64, 8), (9, 6000, 256, 4), (70, 3000, 96, 2)])
def test_decode_shares(dev, n, longest, d, hkv):
    # ragged batches whose tiles are shared by many workgroups: shares that begin and end anywhere in a sequence, also right
    # behind its beginning, empty sequences and ones of a position between them
    r = random.Random(n)
    for seed in range(3):
        lens = [r.choice([0, 1, 32, 33, r.randint(1, longest), r.randint(1, longest)]) for _ in range(n)]
        decode_check(dev, (BF16, F16)[seed % 2], 2 * hkv, hkv, d, 16, lens, seed=seed, quiet=seed > 0)


@pytest.mark.parametrize("room", [1, 1024, 1040, 9000])
@pytest.mark.parametrize("hq,hkv,d", [(8, 2, 128), (3, 3, 64), (12, 2, 256), (20, 1, 96)])
def test_decode_tables(dev, room, hq, hkv, d):
    # what a sequence is divided into depends on the table's width too: whole ones, few pieces, shares that end in a beginning
    for page in (16, 32, 20):
        decode_check(dev, F16, hq, hkv, d, page, [1], room=room, quiet=True)
        decode_check(dev, BF16, hq, hkv, d, page, [1000, 0, 1, 32, 33, 500, 1008], seed=1, room=room)
        decode_check(dev, F16, hq, hkv, d, page, [(61 * i) % 170 for i in range(90)], seed=2, room=room, quiet=True)


def test_decode_many_sequences(dev):
    decode_check(dev, BF16, 4, 2, 64, 16, [(37 * i) % 97 for i in range(150)], quiet=True)


@pytest.mark.parametrize("gain", [8.0, 60.0])
def test_decode_peaked_softmax(dev, gain):
    decode_check(dev, F16, 4, 2, 128, 16, [190, 1000], gain=gain)
    decode_check(dev, BF16, 4, 2, 64, 16, [190, 1000], gain=gain)


@pytest.mark.parametrize("d", [64, 96, 128, 256])
def test_decode_outlier_channel(dev, d):
    # one query element far above the rest: what is small beside it still counts
    for outlier in (30.0, 1000.0):
        decode_check(dev, BF16, 4, 2, d, 16, [300], outlier=outlier, scale=0.01)
        decode_check(dev, F16, 4, 2, d, 16, [300], outlier=outlier, scale=0.01)


def test_decode_absent_pages(dev):
    for page in (16, 7):
        decode_check(dev, BF16, 4, 2, 128, page, [100, 40, 16], absent=[(0, 1), (0, 2), (1, 0), (2, 0), (2, 1), (2, 2)][:5 if page == 7 else 4])


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("d", [32, 40, 64, 96, 128, 200, 256])
def test_scores(dev, dtype, d):
    # sequences of one position: the log-sum-exp is the score.  Products and their sums over 32 elements are exact; pieces
    # of 5 bits and blocks are added in float32: 2^-24 of what is there at each of up to 10 additions, and the scale's rounding
    g = gen(dev, d)
    n = 64
    cache = spa.new_kv_cache(n, 16, 1, d, dtype, "mxfp4", dev)
    held = M.fill(cache, g, dtype)
    q = torch.randn((n, 2, d), generator=g, device=dev)
    q[::3, :, 1] *= 300.0
    q = q.to(dtype)
    table = torch.arange(n, dtype=I32, device=dev)[:, None]
    out, lse = spa.attention_decode(q, cache, table, torch.ones(n, dtype=I32, device=dev), scale=1.0, want_lse=True)
    k = held[0][:, 0, 0]
    want = (q.double() * k[:, None]).sum(-1)
    size = (q.double() * k[:, None]).abs().sum(-1)
    hold = torch.stack([query_error(q[i:i + 1], k[i][None, None], 1.0)[0] for i in range(n)])
    bound = hold + 14 * 2.0 ** -24 * size + 2.0 ** -22 * want.abs() + 2.0 ** -22
    err = (lse.double() - want).abs()
    assert (err <= bound).all(), (err / bound).max().item()
    assert torch.equal(out, held[1][:, 0, 0].to(dtype)[:, None].expand(-1, 2, -1))      # a weight of 1


def test_what_does_not_count_is_not_read(dev):
    # NaN groups past the end, on absent pages' stand-in, in other heads and in other sequences change nothing
    g = gen(dev, 9)
    for page, dtype, d in ((16, BF16, 128), (16, F16, 96), (7, BF16, 64)):
        lens = [37, 5]
        cache = spa.new_kv_cache(12, page, 2, d, dtype, "mxfp4", dev)
        M.fill(cache, g, dtype)
        table = torch.tensor([[3, 4, 5, 6, 7, 8], [9, -1, -1, -1, -1, -1]], dtype=I32, device=dev)
        q = torch.randn((2, 4, d), generator=g, device=dev).to(dtype)
        ln = torch.tensor(lens, dtype=I32, device=dev)
        want = spa.attention_decode(q, cache, table, ln, want_lse=True)
        want = [x.clone() for x in want]
        for s in (cache.k_scale, cache.v_scale):
            s[0] = 255                                          # the page that stands in
            s[table[0, 37 // page].long(), :, :, 37 % page:] = 255
            s[9, :, :, 5:] = 255
        cache.k_scale[11], cache.v_scale[11] = 255, 255
        got = spa.attention_decode(q, cache, table, ln, want_lse=True)
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_nonfinite_values_that_count(dev):
    g = gen(dev, 11)
    for page, d in ((16, 128), (7, 64)):
        cache = spa.new_kv_cache(8, page, 1, d, BF16, "mxfp4", dev)
        M.fill(cache, g, BF16)
        table = torch.arange(8, dtype=I32, device=dev)[None]
        q = torch.randn((1, 2, d), generator=g, device=dev).to(BF16)
        ln = torch.tensor([40], dtype=I32, device=dev)
        clean, _ = spa.attention_decode(q, cache, table, ln)
        cache.v_scale[1, 0, 1, 2] = 255                         # dimensions 32..63 of one value
        out, lse = spa.attention_decode(q, cache, table, ln, want_lse=True)
        assert torch.isnan(out[..., 32:64]).all() and torch.isfinite(lse).all()
        assert torch.equal(out[..., :32], clean[..., :32]) and torch.equal(out[..., 64:], clean[..., 64:])
        cache.k_scale[2, 0, 0, 1] = 255                         # a key: the whole row
        out, lse = spa.attention_decode(q, cache, table, ln, want_lse=True)
        assert torch.isnan(out).all() and torch.isnan(lse).all()
        M.fill(cache, g, BF16)
        for bad in (math.nan, math.inf):                        # a query: its own head alone
            x = q.clone()
            x[0, 1, 3] = bad
            want, _ = spa.attention_decode(q, cache, table, ln)
            out, lse = spa.attention_decode(x, cache, table, ln, want_lse=True)
            assert torch.isnan(out[0, 1]).all() and torch.isnan(lse[0, 1]) and torch.equal(out[0, 0], want[0, 0])


def test_strided_queries_and_given_outputs(dev):
    g = gen(dev, 4)
    cache = spa.new_kv_cache(6, 16, 2, 128, BF16, "mxfp4", dev)
    M.fill(cache, g, BF16)
    x = torch.randn((3, 8 + 4, 128), generator=g, device=dev).to(BF16)
    table = torch.tensor([[0, 1], [2, 3], [4, 5]], dtype=I32, device=dev)
    ln = torch.tensor([20, 32, 1], dtype=I32, device=dev)
    want, _ = spa.attention_decode(x[:, :8].contiguous(), cache, table, ln)
    out = torch.empty_like(want)
    got, _ = spa.attention_decode(x[:, :8], cache, table, ln, out=out)
    assert got is out and torch.equal(got, want)


def test_range_of_exponents(dev):
    # values whose scales differ by 2^60 in one sequence; keys far below and above one
    for dtype, far in ((BF16, 60), (F16, 20)):
        g = gen(dev, far)
        cache = spa.new_kv_cache(4, 16, 1, 128, dtype, "mxfp4", dev)
        held = M.fill(cache, g, dtype)
        cache.v_scale[::2] -= far
        held[1] = M.values(cache.v, cache.v_scale)
        table = torch.arange(4, dtype=I32, device=dev)[None]
        q = torch.randn((1, 4, 128), generator=g, device=dev).to(dtype)
        out, lse = spa.attention_decode(q, cache, table, torch.tensor([64], dtype=I32, device=dev), want_lse=True)
        k, v = (y.permute(0, 2, 1, 3).reshape(64, 1, 128) for y in held)
        r = A.reference(q, k, v, 128 ** -0.5, torch.ones((1, 64), dtype=torch.bool, device=dev))
        r["ds"] = r["ds"] + query_error(q, k, 128 ** -0.5)
        A.check(out, lse, r, dtype, codes=True)


def test_offsets_past_32_bits(dev):
    # codes past 4 GiB and scales past 2 GiB
    page, h, d = 16, 8, 256
    n_pages = (2 ** 31 - 1) // (page * h * 8)                   # 2^28 cells of 128 bytes
    pages = [torch.empty((n_pages, h, page, d // 2), dtype=torch.uint8, device=dev) for _ in range(2)]
    scales = [torch.empty((n_pages, h, d // 32, page), dtype=torch.uint8, device=dev) for _ in range(2)]
    cache = spa.KvCache(*pages, *scales)
    last = n_pages - 3
    g = gen(dev, 2)
    x = torch.randn((2 * page, 2 * h, d), generator=g, device=dev).to(BF16)
    table = torch.tensor([[last, last + 2]], dtype=I32, device=dev)
    pos = torch.arange(2 * page, device=dev)
    slots = (table[0, pos // page].long() * page + pos % page).to(I32)
    spa.kv_write(x[:, :h], x[:, h:], slots, cache)
    small = spa.new_kv_cache(2, page, h, d, BF16, "mxfp4", dev)
    near = torch.tensor([[0, 1]], dtype=I32, device=dev)
    spa.kv_write(x[:, :h], x[:, h:], pos.to(I32), small)
    cu, ln = torch.tensor([0, 30], dtype=I32, device=dev), torch.tensor([30], dtype=I32, device=dev)
    q = torch.randn((1, 16, d), generator=g, device=dev).to(BF16)
    for a, b in zip(spa.kv_read(cache, table, cu, 30, dtype=BF16), spa.kv_read(small, near, cu, 30, dtype=BF16)):
        assert torch.equal(a, b)
    assert torch.equal(spa.attention_decode(q, cache, table, ln)[0], spa.attention_decode(q, small, near, ln)[0])


def test_captured_calls_follow_later_lengths(dev):
    g = gen(dev, 6)
    cache = spa.new_kv_cache(40, 16, 2, 128, BF16, "mxfp4", dev)
    M.fill(cache, g, BF16)
    table = torch.randperm(40, generator=g, device=dev).to(I32).view(2, 20)
    q = torch.randn((2, 8, 128), generator=g, device=dev).to(BF16)
    kv = torch.randn((2, 4, 128), generator=g, device=dev).to(BF16)
    ln, slots = torch.tensor([5, 17], dtype=I32, device=dev), torch.tensor([-1, -1], dtype=I32, device=dev)
    out = torch.empty_like(q)

    def step():
        spa.kv_write(kv[:, :2], kv[:, 2:], slots, cache)
        spa.attention_decode(q, cache, table, ln, out=out)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for lens in ([1, 1], [300, 320], [0, 16], [33, 250]):
        ln.copy_(torch.tensor(lens, dtype=I32))
        slots.copy_(torch.stack([table[s, max(x - 1, 0) // 16] * 16 + max(x - 1, 0) % 16 for s, x in enumerate(lens)]))
        graph.replay()
        torch.cuda.synchronize()
        got = out.clone()
        step()
        assert torch.equal(got, out), lens


def test_calls_on_two_streams(dev):
    g = gen(dev, 8)
    lens = [9000, 40, 3000]
    cache = spa.new_kv_cache(800, 16, 2, 128, F16, "mxfp4", dev)
    M.fill(cache, g, F16)
    table = table_for(dev, g, lens, 16, 800)
    ln = torch.tensor(lens, dtype=I32, device=dev)
    qs = [torch.randn((3, 8, 128), generator=g, device=dev).to(F16) for _ in range(2)]
    want = [spa.attention_decode(q, cache, table, ln)[0] for q in qs]
    streams = [torch.cuda.Stream() for _ in qs]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(5):
        for i, st in enumerate(streams):
            with torch.cuda.stream(st):
                got[i].append(spa.attention_decode(qs[i], cache, table, ln)[0])
    torch.cuda.synchronize()
    for w, all_of in zip(want, got):
        assert all(torch.equal(w, x) for x in all_of)


@pytest.mark.parametrize("hq,hkv,d", [(8, 2, 128), (8, 1, 96), (20, 1, 64), (2, 2, 256)])
def test_nonfinite_queries_stay_by_themselves(dev, hq, hkv, d):
    # a head's query pieces stand beside the other heads' in the matrix product
    g = gen(dev, 12)
    lens = [700, 40, 33, 1]
    for page in (16, 20):
        cache = spa.new_kv_cache(200, page, hkv, d, BF16, "mxfp4", dev)
        M.fill(cache, g, BF16)
        table = table_for(dev, g, lens, page, 200)
        ln = torch.tensor(lens, dtype=I32, device=dev)
        q = torch.randn((4, hq, d), generator=g, device=dev).to(BF16)
        want = spa.attention_decode(q, cache, table, ln)[0]
        q[0, hq - 1, 3], q[1, 0, d - 1], q[3, 1, d // 2] = math.nan, math.inf, -math.inf
        got = spa.attention_decode(q, cache, table, ln)[0]
        hit = torch.zeros((4, hq), dtype=torch.bool, device=dev)
        hit[0, hq - 1] = hit[1, 0] = hit[3, 1] = True
        assert torch.equal(got[~hit], want[~hit]) and torch.isnan(got[hit]).all()
