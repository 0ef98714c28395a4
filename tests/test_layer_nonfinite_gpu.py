"""Infinities and NaN in keys, values and queries: a row that does not see them is not touched, one that sees them says so."""
import math

import pytest
import torch

import attention_bounds as A

pytestmark = pytest.mark.gpu

spa = pytest.importorskip("activation_sparsification_amd")

BF16, F16 = torch.bfloat16, torch.float16
INF, NAN = math.inf, math.nan


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def offsets(lens):
    return torch.tensor([0] + list(lens)).cumsum(0).to(torch.int32).cuda()


def check_rows(got, got_lse, q, k, v, visible, scale, dtype, codes=False):
    """Rows against the reference on finite values; a visible NaN or infinity of v must appear in its dimension, and only
    there.  k and q are finite, or such that the reference's scores are finite or -inf."""
    hq, hkv = q.shape[1], k.shape[1]
    bad = ~torch.isfinite(v)
    r = A.reference(q, k, v.masked_fill(bad, 0.0), scale, visible)
    seen = visible.double()
    per = hq // hkv

    def marks(which):           # [lq, hq, d]: a row sees such a value in this dimension
        m = torch.stack([seen @ which[:, h].double() for h in range(hkv)], 1) > 0
        return m.repeat_interleave(per, 1)

    plus, minus, nan = marks(v == INF), marks(v == -INF), marks(v.isnan())
    nan = nan | (plus & minus)
    plus, minus = plus & ~nan, minus & ~nan
    assert got[nan].isnan().all(), "a visible NaN was lost"
    assert (got[plus] == INF).all() and (got[minus] == -INF).all(), "a visible infinity was lost or became NaN"
    rest = ~(nan | plus | minus)
    A.check(torch.where(rest, got.double(), r["out"]), got_lse, r, dtype, codes)


# ---------------------------------------------------------------------------------------------------------------
# prompts
# ---------------------------------------------------------------------------------------------------------------
def prompt(dtype, hq, hkv, d, lens_q, lens_k, causal, bad, seed=0):
    """bad: (sequence, position, dimensions, value of k or None, value of v or None)."""
    print(f"[prompt] {dtype} heads {hq}/{hkv}x{d} q {lens_q} k {lens_k} causal {causal}", flush=True)
    g = gen(seed)
    q, k, v = (torch.randn((sum(n), h, d), generator=g, device="cuda").to(dtype)
               for n, h in ((lens_q, hq), (lens_k, hkv), (lens_k, hkv)))
    first = [sum(lens_k[:s]) for s in range(len(lens_k))]
    for s, at, dims, of_k, of_v in bad:
        if of_k is not None:
            k[first[s] + at, :, dims] = of_k
        if of_v is not None:
            v[first[s] + at, :, dims] = of_v
    out, lse = spa.attention_prefill(q, k, v, offsets(lens_q), offsets(lens_k), causal=causal, want_lse=True)
    a = c = 0
    for lq, lk in zip(lens_q, lens_k):
        i, j = torch.arange(lq, device="cuda")[:, None], torch.arange(lk, device="cuda")[None, :]
        visible = (j <= i + lk - lq) if causal else torch.ones((lq, lk), dtype=torch.bool, device="cuda")
        ks = k[c:c + lk].double()
        sick = ~torch.isfinite(ks).all(-1).all(-1)
        hit = (visible & sick).any(-1)                  # rows that see a key with a NaN or an infinity
        if bool(hit.any()):
            assert out[a:a + lq][hit].isnan().all() and lse[a:a + lq][hit].isnan().all()
        ok = ~hit
        check_rows(out[a:a + lq][ok], lse[a:a + lq][ok], q[a:a + lq][ok].double(), ks.masked_fill(~torch.isfinite(ks), 0.0),
                   v[c:c + lk].double(), visible[ok] & ~sick, d ** -0.5, dtype)
        a, c = a + lq, c + lk


ALL, SOME = slice(None), slice(3, 6)


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("d", [64, 128, 256, 40, 96, 160])
@pytest.mark.parametrize("value", [NAN, INF, -INF])
def test_prompt_values_of_hidden_keys(dtype, d, value):
    # later positions of the same sequence, in the tile of the diagonal and in later ones
    prompt(dtype, 4, 2, d, [200], [200], True, [(0, 199, SOME, None, value)], seed=d)
    prompt(dtype, 4, 2, d, [130, 90], [130, 90], True, [(0, 70, ALL, None, value), (1, 33, SOME, None, value)], seed=d + 1)
    prompt(dtype, 2, 2, d, [37], [300], True, [(0, 290, SOME, None, value), (0, 264, SOME, None, value)], seed=d + 2)


@pytest.mark.parametrize("d", [64, 128, 256])
def test_prompt_both_infinities_and_the_last_key(d):
    # the tail past the last key repeats nothing that a row does not see
    prompt(BF16, 4, 2, d, [70], [70], False, [(0, 69, SOME, None, INF)], seed=1)
    prompt(BF16, 4, 2, d, [70], [70], True, [(0, 69, SOME, None, -INF)], seed=2)
    prompt(F16, 4, 2, d, [150], [150], True, [(0, 10, SOME, None, INF), (0, 80, SOME, None, -INF)], seed=3)
    prompt(BF16, 4, 2, d, [5, 1], [1, 65], False, [(0, 0, SOME, None, INF), (1, 64, SOME, None, NAN)], seed=4)


@pytest.mark.parametrize("d", [64, 128, 256])
def test_prompt_divided_keys_with_hidden_values(d):
    assert spa.lib().spa_attention_prefill_workspace_bytes(100, 3000, 1, 4, d) > 0
    prompt(BF16, 4, 2, d, [100], [3000], True, [(0, 2950, SOME, None, NAN)], seed=5)
    prompt(F16, 4, 2, d, [100], [3000], True, [(0, 700, SOME, None, INF), (0, 2999, ALL, None, NAN)], seed=6)


@pytest.mark.parametrize("d", [64, 128, 256, 40])
def test_prompt_hidden_keys(d):
    # NaN and infinities in keys themselves; rows that see one have no softmax
    prompt(BF16, 4, 2, d, [200], [200], True, [(0, 100, slice(1), NAN, None)], seed=7)
    prompt(F16, 4, 2, d, [33], [150], True, [(0, 130, ALL, NAN, NAN)], seed=8)


@pytest.mark.parametrize("d", [64, 128, 40, 96, 160])
def test_prompt_scores_of_minus_infinity(d):
    # a key with an infinite element that every query meets with the other sign weighs nothing
    g = gen(d)
    for lk in (50, 2500):
        q, k, v = (torch.randn((n, 2, d), generator=g, device="cuda").to(BF16) for n in (20, lk, lk))
        q[:, :, 2] = q[:, :, 2].abs() + 0.25
        k[31, :, 2] = -INF
        out, lse = spa.attention_prefill(q, k, v, offsets([20]), offsets([lk]), causal=False, want_lse=True)
        visible = torch.ones((20, lk), dtype=torch.bool, device="cuda")
        visible[:, 31] = False
        kf = k.double()
        kf[31] = 0.0
        A.check(out, lse, A.reference(q, kf, v, d ** -0.5, visible), BF16)


@pytest.mark.parametrize("lk", [40, 3000])
@pytest.mark.parametrize("d", [64, 256])
def test_prompt_rows_of_nan(d, lk):
    # a NaN query has NaN outputs and a NaN log-sum-exp; its neighbours have their own
    g = gen(9)
    q, k, v = (torch.randn((n, 2, d), generator=g, device="cuda").to(BF16) for n in (30, lk, lk))
    q[7, 0, 5] = NAN
    out, lse = spa.attention_prefill(q, k, v, offsets([30]), offsets([lk]), causal=False, want_lse=True)
    assert out[7, 0].isnan().all() and lse[7, 0].isnan()
    q[7, 0], out[7, 0], lse[7, 0] = 0.0, 0.0, 0.0
    r = A.reference(q, k, v, d ** -0.5, torch.ones((30, lk), dtype=torch.bool, device="cuda"))
    r["out"][7, 0] = r["lse"][7, 0] = 0.0
    A.check(out, lse, r, BF16)


# ---------------------------------------------------------------------------------------------------------------
# the cache
# ---------------------------------------------------------------------------------------------------------------
@pytest.mark.parametrize("fmt", ["fp8", "int8"])
@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("d", [8, 40, 128, 256])
def test_write_of_nan_and_infinity(fmt, dtype, d):
    # no value stands for them in 8 bits beside finite ones: the whole vector reads back as NaN, and no other does
    g = gen(d)
    h = 3
    k, v = (torch.randn((9, h, d), generator=g, device="cuda").to(dtype) for _ in range(2))
    good = spa.new_kv_cache(1, 16, h, d, dtype, fmt)
    slots = torch.arange(9, dtype=torch.int32, device="cuda")
    spa.kv_write(k, v, slots, good)
    k[1, 0, d // 2], k[2, 1, 0], k[3, 2, d - 1], v[4, 0], v[5, 1] = NAN, INF, -INF, NAN, INF
    v[6, 2, 1], v[6, 2, 2] = NAN, INF
    cache = spa.new_kv_cache(1, 16, h, d, dtype, fmt)
    spa.kv_write(k, v, slots, cache)
    table = torch.zeros((1, 1), dtype=torch.int32, device="cuda")
    got = spa.kv_read(cache, table, offsets([9]), 9, dtype=dtype)
    want = spa.kv_read(good, table, offsets([9]), 9, dtype=dtype)
    for x, y, cells in ((got[0], want[0], ((1, 0), (2, 1), (3, 2))), (got[1], want[1], ((4, 0), (5, 1), (6, 2)))):
        sick = torch.zeros((9, h), dtype=torch.bool, device="cuda")
        for t, head in cells:
            sick[t, head] = True
        assert x[sick].isnan().all(), "a NaN or an infinity was stored as numbers"
        assert torch.equal(x[~sick], y[~sick])


# ---------------------------------------------------------------------------------------------------------------
# single tokens
# ---------------------------------------------------------------------------------------------------------------
def decode(page, lens, q, k, v, hkv=2, d=64):
    """k, v: lists of [len, hkv, d]; a native cache with the sequences on consecutive pages."""
    need = [-(-x // page) for x in lens]
    cache = spa.new_kv_cache(sum(need) + 1, page, hkv, d, q.dtype)
    table = torch.full((len(lens), max(need)), -1, dtype=torch.int32, device="cuda")
    at = 0
    for s, x in enumerate(lens):
        table[s, :need[s]] = torch.arange(at, at + need[s])
        slots = torch.arange(x, dtype=torch.int32, device="cuda") + at * page
        spa.kv_write(k[s], v[s], slots, cache)
        at += need[s]
    return spa.attention_decode(q, cache, table, torch.tensor(lens, dtype=torch.int32, device="cuda"), want_lse=True)


@pytest.mark.parametrize("page", [16, 7, 1, 24])
@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("value", [NAN, INF, -INF])
def test_decode_nonfinite_values(page, dtype, value):
    # the last position, whose row stands in for the tile's end, and one in the middle
    lens = [37, 70, 3, 2000]
    g = gen(page)
    q = torch.randn((4, 8, 64), generator=g, device="cuda").to(dtype)
    k, v = ([torch.randn((x, 2, 64), generator=g, device="cuda").to(dtype) for x in lens] for _ in range(2))
    for s, at in ((0, 36), (1, 40), (2, 2), (3, 1999)):
        v[s][at, :, 3:6] = value
    out, lse = decode(page, lens, q, k, v)
    for s, x in enumerate(lens):
        check_rows(out[s:s + 1], lse[s:s + 1], q[s:s + 1].double(), k[s].double(), v[s].double(),
                   torch.ones((1, x), dtype=torch.bool, device="cuda"), 0.125, dtype)


@pytest.mark.parametrize("page", [16, 7])
def test_decode_rows_of_nan(page):
    # one sequence that is cut, one that is not, one that is empty
    lens = [3000, 20, 0]
    g = gen(3)
    q = torch.randn((3, 4, 64), generator=g, device="cuda").to(BF16)
    k, v = ([torch.randn((x, 2, 64), generator=g, device="cuda").to(BF16) for x in lens] for _ in range(2))
    q[:, 1, 9] = NAN
    out, lse = decode(page, lens, q, k, v)
    assert out[:2, 1].isnan().all() and lse[:2, 1].isnan().all()
    assert (out[2] == 0).all() and (lse[2] == -INF).all()
    rest = [0, 2, 3]
    for s in range(2):
        r = A.reference(q[s:s + 1].nan_to_num(0.0), k[s], v[s], 0.125, torch.ones((1, lens[s]), dtype=torch.bool, device="cuda"))
        r["out"][:, 1] = r["lse"][:, 1] = 0.0
        a, b = out[s:s + 1].clone(), lse[s:s + 1].clone()
        a[:, 1] = b[:, 1] = 0.0
        A.check(a, b, r, BF16)
