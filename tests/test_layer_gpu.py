"""The cache, attention and norm operators on the GPU against 64-bit plain forms (tests/layer_ref.py)."""
import math

import pytest
import torch

import layer_ref as R

pytestmark = pytest.mark.gpu

spa = pytest.importorskip("activation_sparsification_amd")

BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32
NAMES = {BF16: "bf16", F16: "f16", F32: "f32"}


@pytest.fixture(scope="module")
def dev():
    assert torch.cuda.is_available(), "GPU tests need a device"
    return torch.device("cuda:0")


def gen(dev, seed):
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    return g


def offsets(lens, dev):
    return torch.tensor([0] + list(lens)).cumsum(0).to(torch.int32).to(dev)


# ---------------------------------------------------------------------------------------------------------------
# prompt attention
# ---------------------------------------------------------------------------------------------------------------
def prompt_check(dev, dtype, hq, hkv, d, lens_q, lens_k, causal, seed=0, scale=None, packed=False, gain=1.0):
    print(f"[prompt] {NAMES[dtype]} heads {hq}/{hkv}x{d} q {lens_q} k {lens_k} causal {causal}", flush=True)
    g = gen(dev, seed)
    tq, tk = sum(lens_q), sum(lens_k)
    if packed:
        x = torch.randn((tq, hq + 2 * hkv, d), generator=g, device=dev).to(dtype)
        q, k, v = x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:]
    else:
        q, k, v = (torch.randn((t, h, d), generator=g, device=dev).to(dtype) for t, h in ((tq, hq), (tk, hkv), (tk, hkv)))
        q = (q.float() * gain).to(dtype)
    cu_q, cu_k = offsets(lens_q, dev), offsets(lens_k, dev)
    out, lse = spa.attention_prefill(q, k, v, cu_q, cu_k, causal=causal, scale=scale, want_lse=True)
    sc = d ** -0.5 if scale is None else scale
    a = c = 0
    for lq, lk in zip(lens_q, lens_k):
        i, j = torch.arange(lq, device=dev)[:, None], torch.arange(lk, device=dev)[None, :]
        visible = (j <= i + lk - lq) if causal else torch.ones((lq, lk), dtype=torch.bool, device=dev)
        ref = R.attention(q[a:a + lq].double(), k[c:c + lk].double(), v[c:c + lk].double(), sc, visible)
        if lq:
            vmax = float(v[c:c + lk].abs().max()) if lk else 0.0
            R.check_attention(out[a:a + lq], lse[a:a + lq], ref, dtype, lk, vmax)
        a, c = a + lq, c + lk
    return out, lse


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("hq,hkv,d", [(4, 4, 64), (8, 2, 128), (6, 3, 96), (2, 1, 256), (3, 1, 8), (4, 2, 40), (2, 2, 160)])
def test_prompt_heads(dev, dtype, hq, hkv, d):
    prompt_check(dev, dtype, hq, hkv, d, [129, 1, 70], [129, 1, 70], True, seed=d)
    prompt_check(dev, dtype, hq, hkv, d, [65, 33], [100, 7], False, seed=d + 1)


@pytest.mark.parametrize("lens_q,lens_k", [
    ([1], [1]), ([0, 5, 0], [0, 5, 3]), ([127, 128, 129], [127, 128, 129]), ([1, 1, 1], [64, 65, 500]),
    ([64], [0]),                # no keys at all
    ([200, 3], [70, 2]),        # fewer keys than queries: the first queries see nothing
    ([31, 300], [400, 300]), ([700], [700]), ([256], [1300]),
])
@pytest.mark.parametrize("causal", [True, False])
def test_prompt_lengths(dev, lens_q, lens_k, causal):
    prompt_check(dev, BF16, 4, 2, 64, lens_q, lens_k, causal, seed=len(lens_q))
    prompt_check(dev, F16, 2, 1, 128, lens_q, lens_k, causal, seed=1 + len(lens_q))


@pytest.mark.parametrize("d", [40, 64, 128, 256])
def test_prompt_divided_keys(dev, d):
    # few rows over many keys: a tile's keys are divided and joined; rows that see nothing, pieces that some rows see
    # nothing of, sequences too short to divide
    for dtype, causal in ((BF16, True), (F16, True), (BF16, False)):
        assert spa.lib().spa_attention_prefill_workspace_bytes(305, 3290, 3, 4, d) > 0
        prompt_check(dev, dtype, 4, 2, d, [300, 5, 0], [290, 2900, 100], causal, seed=d)
    prompt_check(dev, BF16, 4, 1, d, [1], [5000], True)


def test_prompt_many_sequences(dev):
    lens = [(7 * i) % 41 for i in range(150)]
    prompt_check(dev, BF16, 2, 2, 64, lens, [x + i % 3 for i, x in enumerate(lens)], True)


@pytest.mark.parametrize("gain", [8.0, 60.0])
def test_prompt_peaked_softmax(dev, gain):
    # scores of hundreds: weights of one and zeros, maxima that rise late
    prompt_check(dev, F16, 4, 4, 128, [190], [190], True, gain=gain)
    prompt_check(dev, BF16, 4, 4, 64, [190], [333], True, gain=gain)


def test_prompt_scale_and_packed_views(dev):
    prompt_check(dev, BF16, 8, 2, 128, [130, 62], [130, 62], True, scale=0.3, packed=True)
    prompt_check(dev, F16, 4, 4, 64, [130, 62], [130, 62], False, scale=0.01, packed=True)


def test_prompt_neighbours_are_not_read(dev):
    # NaN and infinities in other sequences' rows and past the last one
    g = gen(dev, 3)
    lens = [77, 50, 90]
    q, k, v = (torch.randn((sum(lens) + 40, 4, 64), generator=g, device=dev).to(BF16) for _ in range(3))
    cu = offsets(lens, dev)
    want, want_lse = spa.attention_prefill(q, k, v, cu, want_lse=True)
    for x, bad in ((k, math.inf), (v, math.nan), (q, math.nan)):
        x[77:127] = bad
        x[sum(lens):] = bad
    out = torch.full_like(q, 7.0)
    got, got_lse = spa.attention_prefill(q, k, v, cu, want_lse=True, out=out)
    for lo, hi in ((0, 77), (127, 217)):
        assert torch.equal(got[lo:hi], want[lo:hi]) and torch.equal(got_lse[lo:hi], want_lse[lo:hi])
    assert (got[sum(lens):] == 7.0).all()        # rows outside every sequence stay as they were


def test_prompt_is_repeatable(dev):
    a, la = prompt_check(dev, BF16, 8, 2, 128, [300, 17], [310, 900], True)
    b, lb = prompt_check(dev, BF16, 8, 2, 128, [300, 17], [310, 900], True)
    assert torch.equal(a, b) and torch.equal(la, lb)


# ---------------------------------------------------------------------------------------------------------------
# the cache
# ---------------------------------------------------------------------------------------------------------------
def random_cache(dev, g, fmt, dtype, n_pages, page, h, d):
    """A cache filled by torch, and the float64 values it stands for, [n_pages, h, page, d] each."""
    vals = [torch.randn((n_pages, h, page, d), generator=g, device=dev).to(dtype) for _ in range(2)]
    if fmt == "native":
        return spa.KvCache(*vals), [x.double() for x in vals]
    codes, scales, stand = [], [], []
    for x in vals:
        c, s = R.quantise(x, fmt)
        codes.append(c.float().to(R.CODE[fmt]))
        scales.append(s.float())
        stand.append(c * s[..., None])
    return spa.KvCache(*codes, *scales), stand


def table_for(dev, g, lens, page, n_pages):
    """Shuffled pages; unused entries of the table are far out of range."""
    width = max(max(-(-x // page) for x in lens), 1)
    perm = torch.randperm(n_pages, generator=g, device=dev).to(torch.int32)
    table = torch.full((len(lens), width), 2 ** 31 - 1, dtype=torch.int32, device=dev)
    at = 0
    for s, x in enumerate(lens):
        need = -(-x // page)
        table[s, :need] = perm[at:at + need]
        at += need
    return table


def cached_rows(stand, table, s, length, page):
    pos = torch.arange(length, device=table.device)
    pg = table[s, pos // page].long()
    return [x[pg, :, pos % page] for x in stand]


@pytest.mark.parametrize("fmt", ["native", "fp8", "int8"])
@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("t,h,d,page", [(1, 1, 8, 1), (33, 3, 40, 7), (64, 8, 128, 16), (50, 2, 256, 100), (17, 4, 64, 32),
                                        (300, 5, 96, 16)])
def test_kv_write(dev, fmt, dtype, t, h, d, page):
    print(f"[kv_write] {fmt} {NAMES[dtype]} t {t} heads {h}x{d} page {page}", flush=True)
    g = gen(dev, t + d)
    n_pages = -(-t // page) + 3
    cache = spa.new_kv_cache(n_pages, page, h, d, dtype, fmt, dev)
    x = torch.randn((t, 2 * h + 1, d), generator=g, device=dev) * 3
    x[0, 0] = 0.0                                               # a zero vector
    if t > 4:
        x[1, 0] *= 1e-4
        x[2, 0] = 1.0                                           # ties everywhere
        x[3, 0, : d // 2] = 2.0 ** -120 if dtype == BF16 else 0.0
        x[3, 0, d // 2:] = 0.0
    x = x.to(dtype)
    k, v = x[:, :h], x[:, h:2 * h]
    slots = torch.randperm(n_pages * page, generator=g, device=dev)[:t].to(torch.int32)
    skip = torch.rand(t, generator=g, device=dev) < 0.1
    slots[skip] = -1
    if t > 8:
        slots[5], slots[6] = n_pages * page, 2 ** 31 - 1        # past the cache: skipped as well
        skip[5:7] = True
    marked = [b for b in (cache.k, cache.v, cache.k_scale, cache.v_scale) if b is not None]
    for b in marked:
        b.view(torch.uint8).fill_(0x35)
    want = [b.clone() for b in marked]
    spa.kv_write(k, v, slots, cache)
    live = (~skip).nonzero().squeeze(-1)
    pg, off = slots[live].long() // page, slots[live].long() % page
    for i, rows in enumerate((k[live], v[live])):
        if fmt == "native":
            want[i][pg, :, off] = rows
        else:
            c, s = R.quantise(rows, fmt)
            want[i].view(torch.uint8)[pg, :, off] = c.float().to(R.CODE[fmt]).view(torch.uint8)
            want[i + 2][pg, :, off] = s.float()
    for got, ref in zip(marked, want):
        a, b = got.contiguous().view(torch.uint8), ref.contiguous().view(torch.uint8)
        if got.dtype == torch.float8_e4m3fn:                    # the sign of a zero code is free
            a, b = torch.where(a == 0x80, 0, a), torch.where(b == 0x80, 0, b)
        assert torch.equal(a, b)


@pytest.mark.parametrize("fmt", ["native", "fp8", "int8"])
@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("lens,h,d,page", [([1], 1, 8, 1), ([0, 33, 0, 5], 3, 40, 7), ([100, 7], 8, 128, 16), ([77], 2, 256, 100),
                                           ([3 * i % 29 for i in range(140)], 2, 64, 8), ([65, 64], 1, 96, 64)])
def test_kv_read(dev, fmt, dtype, lens, h, d, page):
    print(f"[kv_read] {fmt} {NAMES[dtype]} {len(lens)} sequences heads {h}x{d} page {page}", flush=True)
    g = gen(dev, d)
    n_pages = sum(-(-x // page) for x in lens) + 2
    cache, stand = random_cache(dev, g, fmt, dtype, n_pages, page, h, d)
    table = table_for(dev, g, lens, page, n_pages)
    total = sum(lens)
    k, v = spa.kv_read(cache, table, offsets(lens, dev), total, dtype=dtype)
    want = [cached_rows(stand, table, s, x, page) for s, x in enumerate(lens)]
    for i, got in enumerate((k, v)):
        ref = torch.cat([w[i] for w in want])
        assert got.shape == (total, h, d) and torch.equal(got, R.f32(ref).float().to(dtype))


def test_kv_read_absent_pages_are_zero(dev):
    g = gen(dev, 1)
    cache, stand = random_cache(dev, g, "fp8", BF16, 6, 16, 2, 64)
    table = torch.tensor([[0, -1, 6, 2], [2 ** 31 - 1, 3, -2 ** 31, 4]], dtype=torch.int32, device=dev)
    k, v = spa.kv_read(cache, table, offsets([80, 64], dev), 150, k_out=torch.full((150, 2, 64), 5.0, dtype=BF16, device=dev),
                       v_out=torch.full((150, 2, 64), 5.0, dtype=BF16, device=dev))
    for got, ref in ((k, stand[0]), (v, stand[1])):
        want = torch.zeros((144, 2, 64), dtype=torch.float64, device=dev)
        for row, pg in ((0, 0), (48, 2), (96, 3), (128, 4)):
            want[row:row + 16] = ref[pg].transpose(0, 1)
        assert torch.equal(got[:144], R.f32(want).float().to(BF16))
        assert (got[144:] == 5.0).all()                         # rows of no sequence


@pytest.mark.parametrize("fmt", ["native", "int8"])
def test_offsets_past_32_bits(dev, fmt):
    # pages whose first byte lies past 2^32: written, read back and attended to
    page, h, d = 16, 8, 128
    per = page * h * d * (2 if fmt == "native" else 1)
    n_pages = (2 ** 32 + 2 ** 28) // per
    if torch.cuda.mem_get_info(dev)[0] < 24 << 30:
        pytest.skip("needs 24 GiB of free device memory")
    code = BF16 if fmt == "native" else torch.int8
    pages = [torch.empty((n_pages, h, page, d), dtype=code, device=dev) for _ in range(2)]
    scales = [None if fmt == "native" else torch.empty((n_pages, h, page), device=dev) for _ in range(2)]
    cache = spa.KvCache(*pages, *scales)
    g = gen(dev, 2)
    t = 90
    k, v = (torch.randn((t, h, d), generator=g, device=dev).to(BF16) for _ in range(2))
    table = torch.tensor([[n_pages - 1, 3, n_pages - 2, n_pages // 2, n_pages - 9, 0]], dtype=torch.int32, device=dev)
    pos = torch.arange(t, device=dev)
    spa.kv_write(k, v, (table[0, pos // page].long() * page + pos % page).to(torch.int32), cache)
    rk, rv = spa.kv_read(cache, table, offsets([t], dev), t, dtype=BF16)
    want = []
    for x in (k, v):
        c, s = (x.double(), None) if fmt == "native" else R.quantise(x, fmt)
        want.append(c if s is None else c * s[..., None])
    for got, ref in ((rk, want[0]), (rv, want[1])):
        assert torch.equal(got, R.f32(ref).float().to(BF16))
    q = torch.randn((1, 16, d), generator=g, device=dev).to(BF16)
    out, lse = spa.attention_decode(q, cache, table, torch.tensor([t], dtype=torch.int32, device=dev), want_lse=True)
    ref = R.attention(q.double(), want[0], want[1], d ** -0.5, torch.ones((1, t), dtype=torch.bool, device=dev))
    R.check_attention(out, lse, ref, BF16, t, 6.0)


# ---------------------------------------------------------------------------------------------------------------
# decode attention
# ---------------------------------------------------------------------------------------------------------------
def decode_check(dev, dtype, fmt, hq, hkv, d, page, lens, seed=0, scale=None, gain=1.0):
    print(f"[decode] {NAMES[dtype]} {fmt} heads {hq}/{hkv}x{d} page {page} lens {lens[:8]}", flush=True)
    g = gen(dev, seed)
    n_pages = sum(-(-x // page) for x in lens) + 3
    cache, stand = random_cache(dev, g, fmt, dtype, n_pages, page, hkv, d)
    table = table_for(dev, g, lens, page, n_pages)
    q = (torch.randn((len(lens), hq, d), generator=g, device=dev) * gain).to(dtype)
    ln = torch.tensor(lens, dtype=torch.int32, device=dev)
    out, lse = spa.attention_decode(q, cache, table, ln, scale=scale, want_lse=True)
    for s, x in enumerate(lens):
        k, v = cached_rows(stand, table, s, x, page)
        ref = R.attention(q[s:s + 1].double(), k, v, d ** -0.5 if scale is None else scale,
                          torch.ones((1, x), dtype=torch.bool, device=dev))
        R.check_attention(out[s:s + 1], lse[s:s + 1], ref, dtype, x, float(v.abs().max()) if x else 0.0)
    return out, lse


@pytest.mark.parametrize("fmt", ["native", "fp8", "int8"])
@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("hq,hkv,d", [(32, 8, 128), (4, 4, 64), (16, 1, 128), (17, 1, 64), (40, 1, 128), (6, 3, 96), (2, 1, 256),
                                      (3, 1, 8), (8, 2, 40), (20, 2, 200)])
def test_decode_heads(dev, fmt, dtype, hq, hkv, d):
    decode_check(dev, dtype, fmt, hq, hkv, d, 16, [1, 0, 37, 200], seed=d + hq)


@pytest.mark.parametrize("fmt", ["native", "fp8", "int8"])
@pytest.mark.parametrize("page", [1, 7, 16, 32, 64, 100])
def test_decode_pages_and_lengths(dev, fmt, page):
    decode_check(dev, BF16, fmt, 8, 2, 64, page, [31, 32, 33, 63, 64, 65, 127, 128, 129, 1, 0, 500], seed=page)


@pytest.mark.parametrize("fmt", ["native", "fp8", "int8"])
def test_decode_long_and_split(dev, fmt):
    decode_check(dev, BF16, fmt, 8, 2, 128, 16, [20011, 3, 4097], seed=1)
    decode_check(dev, F16, fmt, 4, 1, 64, 32, [60001], seed=2)


def test_decode_many_sequences(dev):
    decode_check(dev, BF16, "native", 4, 2, 64, 8, [(13 * i) % 97 for i in range(200)], seed=3)


def test_decode_long_among_short(dev):
    # more sequences than a wave has lanes, and one that is cut many times in the middle of them
    decode_check(dev, BF16, "fp8", 4, 2, 128, 16, [5] * 70 + [20000] + [0, 33] * 3, seed=5)
    decode_check(dev, F16, "native", 4, 2, 64, 7, [5] * 70 + [3000] + [0, 33] * 3, seed=6)


def test_decode_more_sequences_than_pieces(dev):
    decode_check(dev, F16, "fp8", 8, 8, 64, 16, [(31 * i) % 300 for i in range(400)], seed=4)


@pytest.mark.parametrize("fmt", ["native", "int8"])
def test_decode_peaked_softmax(dev, fmt):
    decode_check(dev, F16, fmt, 8, 2, 128, 16, [700, 90], seed=5, gain=40.0)
    decode_check(dev, BF16, fmt, 8, 2, 128, 16, [700, 90], seed=6, scale=2.0)


@pytest.mark.parametrize("fmt", ["native", "fp8", "int8"])
def test_decode_reads_no_hidden_position(dev, fmt):
    # NaN in every cell that no sequence counts: page tails, spare pages, the pages of absent entries
    g = gen(dev, 8)
    page, h, d, lens = 16, 2, 128, [37, 300, 16, 5]
    n_pages = 40
    cache, stand = random_cache(dev, g, fmt, BF16, n_pages, page, h, d)
    table = table_for(dev, g, lens, page, n_pages)
    ln = torch.tensor(lens, dtype=torch.int32, device=dev)
    q = torch.randn((4, 8, d), generator=g, device=dev).to(BF16)
    table[1, 3], table[1, 7], table[3, 0] = -1, n_pages, -7          # absent pages: 3 has nothing left
    used = torch.zeros((n_pages, page), dtype=torch.bool, device=dev)
    for s, x in enumerate(lens):
        for p in range(x):
            pg = int(table[s, p // page])
            if 0 <= pg < n_pages:
                used[pg, p % page] = True
    hidden = (~used)[:, None, :].expand(n_pages, h, page)
    if fmt != "int8":
        for x in (cache.k, cache.v):
            x.view(torch.uint8 if fmt == "fp8" else torch.int16)[hidden] = 0x7F if fmt == "fp8" else 0x7FC0
    for x in (cache.k_scale, cache.v_scale):
        if x is not None:
            x[hidden] = math.nan
    out, lse = spa.attention_decode(q, cache, table, ln, want_lse=True)
    for s, x in enumerate(lens):
        pos = torch.tensor([p for p in range(x) if 0 <= int(table[s, p // page]) < n_pages], dtype=torch.long, device=dev)
        pg = table[s, pos // page].long()
        k, v = (y[pg, :, pos % page] for y in stand)
        ref = R.attention(q[s:s + 1].double(), k, v, d ** -0.5, torch.ones((1, len(pos)), dtype=torch.bool, device=dev))
        R.check_attention(out[s:s + 1], lse[s:s + 1], ref, BF16, x, 6.0)
    assert (out[3] == 0).all() and (lse[3] == -math.inf).all()


def test_decode_lengths_past_the_table(dev):
    # a length beyond the table's pages counts the pages there are; a negative one counts nothing
    g = gen(dev, 9)
    cache, stand = random_cache(dev, g, "native", BF16, 8, 16, 2, 64)
    table = torch.tensor([[1, 2], [3, 4]], dtype=torch.int32, device=dev)
    q = torch.randn((2, 4, 64), generator=g, device=dev).to(BF16)
    a, la = spa.attention_decode(q, cache, table, torch.tensor([10 ** 9, -5], dtype=torch.int32, device=dev), want_lse=True)
    b, lb = spa.attention_decode(q, cache, table, torch.tensor([32, 0], dtype=torch.int32, device=dev), want_lse=True)
    assert torch.equal(a, b) and torch.equal(la, lb) and (a[1] == 0).all()


def test_decode_strided_queries_and_repeatability(dev):
    g = gen(dev, 10)
    cache, _ = random_cache(dev, g, "fp8", BF16, 300, 16, 2, 128)
    lens = [3000, 700]
    table = table_for(dev, g, lens, 16, 300)
    ln = torch.tensor(lens, dtype=torch.int32, device=dev)
    x = torch.randn((2, 12, 128), generator=g, device=dev).to(BF16)
    a, la = spa.attention_decode(x[:, :8], cache, table, ln, want_lse=True)
    for _ in range(3):
        b, lb = spa.attention_decode(x[:, :8].contiguous(), cache, table, ln, want_lse=True)
        assert torch.equal(a, b) and torch.equal(la, lb)


def test_decode_in_a_graph_follows_the_lengths(dev):
    g = gen(dev, 11)
    cache, _ = random_cache(dev, g, "int8", BF16, 400, 16, 2, 128)
    lens = [3000, 700, 0]
    table = table_for(dev, g, [3000, 2000, 1000], 16, 400)
    ln = torch.tensor(lens, dtype=torch.int32, device=dev)
    q = torch.randn((3, 8, 128), generator=g, device=dev).to(BF16)
    out = torch.empty_like(q)
    ws = torch.empty(spa.lib().spa_attention_decode_workspace_bytes(3, 8, 2, 128), dtype=torch.uint8, device=dev)
    spa.attention_decode(q, cache, table, ln, out=out, ws=ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        spa.attention_decode(q, cache, table, ln, out=out, ws=ws)
    for step, now in enumerate(([3000, 700, 0], [1, 2000, 999], [0, 0, 0], [2999, 1, 1000])):
        ln.copy_(torch.tensor(now, dtype=torch.int32))
        q.mul_(0.9)
        want, _ = spa.attention_decode(q, cache, table, ln)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want), step


def test_calls_on_another_stream(dev):
    g = gen(dev, 12)
    lens = [900, 33]
    q, k, v = (torch.randn((sum(lens), h, 128), generator=g, device=dev).to(BF16) for h in (8, 2, 2))
    cu = offsets(lens, dev)
    ln = torch.tensor(lens, dtype=torch.int32, device=dev)
    table = table_for(dev, g, lens, 16, 80)
    pos = [torch.arange(x, device=dev) for x in lens]
    slots = torch.cat([table[s, p // 16].long() * 16 + p % 16 for s, p in enumerate(pos)]).to(torch.int32)
    last = cu[1:].long() - 1
    w = torch.ones(256, dtype=BF16, device=dev)

    def chain():
        cache = spa.new_kv_cache(80, 16, 2, 128, BF16, "fp8", dev)
        spa.kv_write(k, v, slots, cache)
        rk, rv = spa.kv_read(cache, table, cu, sum(lens), dtype=BF16)
        a, _ = spa.attention_prefill(q, rk, rv, cu)
        b, _ = spa.attention_decode(q[last], cache, table, ln)
        h, y = spa.gated_residual_norm(a.view(-1, 256), None, pre_weight=w)
        return a, b, h, y

    want = chain()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        torch.cuda._sleep(2_000_000)
        got = chain()
    side.synchronize()
    for x, y in zip(got, want):
        assert torch.equal(x, y)
    # the last prompt row and the decode call see the same keys
    assert (got[0][last].double() - got[1].double()).abs().max() < 2.0 ** -5


# ---------------------------------------------------------------------------------------------------------------
# norms
# ---------------------------------------------------------------------------------------------------------------
def norm_check(dev, dtype, stream, t, c, post, pre, gate, weights=True, offset=0.0, eps=1e-5, seed=0, residual=True):
    print(f"[norm] {NAMES[dtype]}/{NAMES[stream]} [{t}, {c}] {post}->{pre} gate {gate}", flush=True)
    g = gen(dev, seed + c)
    x = (torch.randn((t, c), generator=g, device=dev) + offset).to(dtype)
    res = (torch.randn((t, c), generator=g, device=dev) * 2).to(stream) if residual else None
    par = {}
    for which, kind in (("post", post), ("pre", pre)):
        par[which + "_weight"] = (1 + torch.randn(c, generator=g, device=dev) / 4).to(dtype) if weights and kind != "none" else None
        par[which + "_bias"] = (torch.randn(c, generator=g, device=dev) / 8).to(dtype) if weights and kind == "layer" else None
    gt = {"none": None, "channel": (c,), "token": (t, c)}[gate]
    gt = None if gt is None else torch.randn(gt, generator=g, device=dev).to(dtype)
    h, y = spa.gated_residual_norm(x, res, post=post, pre=pre, gate=gt, scale=-0.75, eps=eps, **par)
    u, us = R.norm(x.double(), post, par["post_weight"], par["post_bias"], eps)
    gd = 1.0 if gt is None else gt.double()
    rd = torch.zeros_like(u) if res is None else res.double()
    hd = rd - 0.75 * gd * u
    h_size = rd.abs() + 0.75 * (us * gd if gt is None else us * gd.abs())
    yd, ys = R.norm(hd, pre, par["pre_weight"], par["pre_bias"], eps)
    # y's terms see h's float32 error through the same factor as h itself; the row's largest covers the shared mean
    # and root
    grow = h_size.amax(-1, keepdim=True) / (hd.abs().amax(-1, keepdim=True) + 1e-30)
    out_t = dtype if residual is False else stream
    for got, ref, size, ty in ((h, hd, h_size, out_t), (y, yd, ys + ys.amax(-1, keepdim=True) * grow, dtype)):
        assert got.dtype == ty and got.shape == ref.shape
        err, bound = (got.double() - ref).abs(), R.U[ty] * ref.abs() + 2.0 ** -17 * size + 2.0 ** -24
        assert (err <= bound).all(), f"error {(err / bound).max().item():.3f} of its bound"


@pytest.mark.parametrize("dtype,stream", [(BF16, BF16), (BF16, F32), (F16, F16), (F16, F32), (F32, F32)])
@pytest.mark.parametrize("t,c", [(1, 1), (3, 7), (2, 8), (5, 520), (4, 1000), (1, 4096), (3, 4097), (2, 8200), (2, 16384),
                                 (1, 20001), (2, 33000), (1, 65536)])
def test_norm_sizes(dev, dtype, stream, t, c):
    norm_check(dev, dtype, stream, t, c, "rms", "rms", "channel")
    norm_check(dev, dtype, stream, t, c, "layer", "layer", "token", seed=1)


@pytest.mark.parametrize("t,c", [(1500, 4096), (9000, 8), (3000, 512), (2100, 1000), (700, 9), (300, 16384)])
def test_norm_many_rows(dev, t, c):
    # more rows than workgroups on the chip: each walks over several
    norm_check(dev, BF16, F32, t, c, "rms", "layer", "token")
    norm_check(dev, F16, F16, t, c, "layer", "rms", "channel")


@pytest.mark.parametrize("post", ["none", "rms", "layer"])
@pytest.mark.parametrize("pre", ["none", "rms", "layer"])
@pytest.mark.parametrize("gate", ["none", "channel", "token"])
def test_norm_kinds(dev, post, pre, gate):
    norm_check(dev, BF16, F32, 9, 768, post, pre, gate)
    norm_check(dev, F16, F16, 9, 776, post, pre, gate, weights=False, residual=False)


def test_norm_far_from_zero(dev):
    # a mean a thousand times the spread: the variance is taken about it
    norm_check(dev, F32, F32, 4, 4096, "layer", "layer", "none", offset=1000.0)


def test_norm_zero_rows_and_eps(dev):
    x = torch.zeros((3, 512), dtype=BF16, device=dev)
    for kind in ("rms", "layer"):
        h, y = spa.gated_residual_norm(x, None, post=kind, pre=kind)
        assert (h == 0).all() and (y == 0).all()


def test_norm_in_place(dev):
    g = gen(dev, 5)
    x, w = torch.randn((6, 4096), generator=g, device=dev).to(BF16), torch.randn(4096, generator=g, device=dev).to(BF16)
    res = torch.randn((6, 4096), generator=g, device=dev)
    want = spa.gated_residual_norm(x, res, post="rms", post_weight=w, gate=w, pre="layer")
    got = spa.gated_residual_norm(x, res, post="rms", post_weight=w, gate=w, pre="layer", h_out=res, y_out=x)
    assert got[0] is res and got[1] is x and torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_empty_calls(dev):
    e = torch.empty((0, 64), dtype=BF16, device=dev)
    h, y = spa.gated_residual_norm(e, e)
    assert h.shape == y.shape == (0, 64)
    cache = spa.new_kv_cache(2, 16, 2, 64, BF16, "fp8", dev)
    none = torch.empty((0,), dtype=torch.int32, device=dev)
    r = torch.empty((0, 2, 64), dtype=BF16, device=dev)
    spa.kv_write(r, r, none, cache)
    k, v = spa.kv_read(cache, torch.zeros((1, 1), dtype=torch.int32, device=dev), offsets([0], dev), 0, dtype=BF16)
    assert k.shape == v.shape == (0, 2, 64)
    out, lse = spa.attention_decode(r, cache, torch.zeros((0, 1), dtype=torch.int32, device=dev), none, want_lse=True)
    assert out.shape == (0, 2, 64) and lse.shape == (0, 2)
    out, _ = spa.attention_prefill(r, r, r, offsets([], dev))
    assert out.shape == (0, 2, 64)
    q = torch.ones((1, 2, 64), dtype=BF16, device=dev)
    out, lse = spa.attention_decode(q, cache, torch.empty((1, 0), dtype=torch.int32, device=dev),
                                    torch.ones(1, dtype=torch.int32, device=dev), want_lse=True)
    assert (out == 0).all() and (lse == -math.inf).all()


# ---------------------------------------------------------------------------------------------------------------
# refusals
# ---------------------------------------------------------------------------------------------------------------
def test_refusals(dev):
    i32 = torch.int32
    q, kv = torch.zeros((4, 8, 64), dtype=BF16, device=dev), torch.zeros((4, 2, 64), dtype=BF16, device=dev)
    cu, table, ln = offsets([4], dev), torch.zeros((4, 1), dtype=i32, device=dev), torch.ones(4, dtype=i32, device=dev)
    cache = spa.new_kv_cache(2, 16, 2, 64, BF16, "native", dev)
    slots = torch.arange(4, dtype=i32, device=dev)
    with pytest.raises(ValueError):
        spa.attention_prefill(q.cpu(), kv, kv, cu)
    with pytest.raises(ValueError):
        spa.attention_prefill(q, kv.half(), kv, cu)
    with pytest.raises(ValueError):
        spa.attention_prefill(q, kv, kv, cu.long())
    with pytest.raises(ValueError):
        spa.attention_prefill(q, kv, kv, cu, out=torch.empty((4, 8, 32), dtype=BF16, device=dev))
    with pytest.raises(ValueError):
        spa.attention_prefill(q.transpose(1, 2), kv, kv, cu)                     # last axis not dense
    for bad, status in ((dict(scale=0.0), 1), (dict(scale=math.nan), 1), (dict(scale=math.inf), 1)):
        with pytest.raises(spa.SpaError) as e:
            spa.attention_prefill(q, kv, kv, cu, **bad)
        assert e.value.status == status
    with pytest.raises(spa.SpaError) as e:                                       # 8 query heads, 3 key-value heads
        spa.attention_prefill(q, torch.zeros((4, 3, 64), dtype=BF16, device=dev), torch.zeros((4, 3, 64), dtype=BF16, device=dev), cu)
    assert e.value.status == 1
    with pytest.raises(spa.SpaError) as e:                                       # float32 vectors
        spa.attention_prefill(q.float(), kv.float(), kv.float(), cu)
    assert e.value.status == 2
    with pytest.raises(spa.SpaError) as e:                                       # head_dim not whole 16-byte pieces
        x = torch.zeros((4, 2, 60), dtype=BF16, device=dev)
        spa.attention_prefill(x, x, x, cu)
    assert e.value.status == 2
    with pytest.raises(spa.SpaError) as e:                                       # rows that start off 16 bytes
        x = torch.zeros((4, 2 * 64 + 4), dtype=BF16, device=dev)[:, 4:].unflatten(1, (2, 64))
        spa.attention_prefill(x, x, x, cu)
    assert e.value.status == 2
    with pytest.raises(ValueError):
        spa.KvCache(cache.k, cache.v, torch.zeros((2, 2, 16), device=dev), torch.zeros((2, 2, 16), device=dev))
    with pytest.raises(ValueError):
        spa.KvCache(cache.k.to(torch.int8), cache.v.to(torch.int8))
    with pytest.raises(ValueError):
        spa.KvCache(cache.k.transpose(1, 2), cache.v.transpose(1, 2))
    with pytest.raises(ValueError):
        spa.kv_write(kv.half(), kv.half(), slots, cache)
    with pytest.raises(ValueError):
        spa.kv_write(kv, kv, slots[:3], cache)
    with pytest.raises(ValueError):
        spa.kv_write(torch.zeros((4, 3, 64), dtype=BF16, device=dev), torch.zeros((4, 3, 64), dtype=BF16, device=dev), slots, cache)
    with pytest.raises(ValueError):
        spa.attention_decode(q, cache, table.long(), ln)
    with pytest.raises(ValueError):
        spa.attention_decode(q, cache, table, ln[:3])
    with pytest.raises(spa.SpaError) as e:
        spa.attention_decode(q, cache, table, ln, ws=torch.empty(16, dtype=torch.uint8, device=dev))
    assert e.value.status == 1
    with pytest.raises(spa.SpaError) as e:
        spa.attention_decode(q, cache, table, ln, scale=-1.0)
    assert e.value.status == 1
    with pytest.raises(ValueError):
        spa.kv_read(spa.new_kv_cache(2, 16, 2, 64, BF16, "int8", dev), table, offsets([1, 1, 1, 1], dev), 4)
    x = torch.zeros((4, 64), dtype=BF16, device=dev)
    with pytest.raises(ValueError):
        spa.gated_residual_norm(x, x, post="batch")
    with pytest.raises(ValueError):
        spa.gated_residual_norm(x, x[:3])
    with pytest.raises(ValueError):
        spa.gated_residual_norm(x, x, gate=torch.zeros((3, 64), dtype=BF16, device=dev))
    with pytest.raises(spa.SpaError) as e:                                       # residual stream narrower than the block
        spa.gated_residual_norm(x.float(), x)
    assert e.value.status == 2
    with pytest.raises(spa.SpaError) as e:
        spa.gated_residual_norm(x, x, eps=-1.0)
    assert e.value.status == 1
    with pytest.raises(spa.SpaError) as e:
        y = torch.zeros((1, 65544), dtype=BF16, device=dev)
        spa.gated_residual_norm(y, y)
    assert e.value.status == 2
