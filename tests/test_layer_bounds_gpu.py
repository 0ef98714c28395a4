"""Attention against bounds that small values, long sequences and single tiles cannot hide behind, and the forms that the C
entries have beside the Python ones."""
import ctypes

import pytest
import torch

import attention_bounds as A

pytestmark = pytest.mark.gpu

spa = pytest.importorskip("activation_sparsification_amd")

BF16, F16, I32 = torch.bfloat16, torch.float16, torch.int32
FORMATS = ["native", "fp8", "int8"]


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def offsets(lens):
    return torch.tensor([0] + list(lens)).cumsum(0).to(I32).cuda()


def prompt(dtype, hq, hkv, d, lens_q, lens_k, causal, size=1.0, gain=1.0, seed=0):
    print(f"[bounds] {dtype} heads {hq}/{hkv}x{d} q {lens_q} k {lens_k} causal {causal} values {size} gain {gain}", flush=True)
    g = gen(seed + d)
    q = (gain * torch.randn((sum(lens_q), hq, d), generator=g, device="cuda")).to(dtype)
    k = torch.randn((sum(lens_k), hkv, d), generator=g, device="cuda").to(dtype)
    v = (size * torch.randn((sum(lens_k), hkv, d), generator=g, device="cuda")).to(dtype)
    out, lse = spa.attention_prefill(q, k, v, offsets(lens_q), offsets(lens_k), causal=causal, want_lse=True)
    a = c = 0
    for lq, lk in zip(lens_q, lens_k):
        i, j = torch.arange(lq, device="cuda")[:, None], torch.arange(lk, device="cuda")[None, :]
        visible = (j <= i + lk - lq) if causal else torch.ones((lq, lk), dtype=torch.bool, device="cuda")
        r = A.reference(q[a:a + lq], k[c:c + lk], v[c:c + lk], d ** -0.5, visible)
        A.check(out[a:a + lq], lse[a:a + lq], r, dtype)
        a, c = a + lq, c + lk


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("hq,hkv,d", [(4, 4, 64), (8, 2, 128), (6, 3, 96), (2, 1, 256), (3, 1, 8), (4, 2, 40), (2, 2, 160),
                                      (17, 1, 72), (4, 2, 248)])
@pytest.mark.parametrize("causal", [True, False])
def test_prompts(dtype, hq, hkv, d, causal):
    prompt(dtype, hq, hkv, d, [129, 1, 70, 0, 300], [129, 1, 200, 5, 300], causal)


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("size,gain", [(1e-3, 1.0), (1e-4, 4.0), (1000.0, 0.1), (1.0, 30.0)])
def test_prompts_of_other_sizes(dtype, size, gain):
    prompt(dtype, 4, 2, 128, [400, 77], [400, 500], True, size, gain)
    prompt(dtype, 4, 2, 64, [33], [4000], True, size, gain)         # divided keys


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("d", [64, 128, 256, 80])
def test_few_rows_over_many_keys(dtype, d):
    assert spa.lib().spa_attention_prefill_workspace_bytes(100, 20000, 1, 4, d) > 0
    prompt(dtype, 4, 2, d, [100], [20000], True)


def test_many_prompts_and_a_long_cached_one():
    prompt(BF16, 4, 2, 64, [40] * 70 + [64] + [3] * 5, [40] * 70 + [6000] + [3] * 5, True)
    prompt(F16, 4, 2, 128, [64] * 9 + [64], [64] * 9 + [9000], True)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("n", [1, 31, 33, 700, 60001])
@pytest.mark.parametrize("hq,hkv,d,page", [(4, 1, 64, 32), (8, 2, 128, 16), (5, 1, 80, 7)])
def test_decode(fmt, dtype, n, hq, hkv, d, page):
    print(f"[bounds] decode {fmt} {dtype} {n} heads {hq}/{hkv}x{d} page {page}", flush=True)
    g = gen(n + d)
    for size in (1.0, 1e-3):
        q, k, v = (torch.randn(s, generator=g, device="cuda") for s in ((1, hq, d), (n, hkv, d), (n, hkv, d)))
        pages = -(-n // page)
        cache = spa.new_kv_cache(pages, page, hkv, d, dtype, fmt)
        spa.kv_write(k.to(dtype), (size * v).to(dtype), torch.arange(n, dtype=I32, device="cuda"), cache)
        table = torch.arange(pages, dtype=I32, device="cuda")[None]
        held = spa.kv_read(cache, table, offsets([n]), n, dtype=dtype)
        if fmt != "native":     # what the codes stand for, not yet rounded to the vectors' type
            held = [(c.float().double() * s.double()[..., None]).transpose(1, 2).reshape(-1, hkv, d)[:n]
                    for c, s in ((cache.k, cache.k_scale), (cache.v, cache.v_scale))]
        q = q.to(dtype)
        out, lse = spa.attention_decode(q, cache, table, torch.tensor([n], dtype=I32, device="cuda"), want_lse=True)
        r = A.reference(q, *held, d ** -0.5, torch.ones((1, n), dtype=torch.bool, device="cuda"))
        A.check(out, lse, r, dtype, codes=fmt != "native")


# ---------------------------------------------------------------------------------------------------------------
# the C entries' own forms
# ---------------------------------------------------------------------------------------------------------------
def ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


@pytest.mark.parametrize("c", [24, 1000, 4096, 9000, 16384, 20001, 40000, 65536])
@pytest.mark.parametrize("rows", [1, 700])
@pytest.mark.parametrize("post,pre", [(0, 1), (1, 0), (2, 2)])
def test_norm_with_one_output(c, rows, post, pre):
    # h or y alone is what the call with both writes, and nothing else is written
    B, L = spa._binding, spa.lib()
    g = gen(c)
    x, w, gate = (torch.randn(s, generator=g, device="cuda").to(BF16) for s in ((rows, c), (c,), (rows, c)))
    res = torch.randn((rows, c), generator=g, device="cuda")
    kinds = ["none", "rms", "layer"]
    both = spa.gated_residual_norm(x, res, post=kinds[post], post_weight=w if post else None, gate=gate, scale=0.5,
                                   pre=kinds[pre], pre_weight=w if pre else None)
    stream = ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
    for h, y in ((torch.full_like(res, 7.0), None), (None, torch.full_like(x, 7.0))):
        st = L.gated_residual_norm(ptr(x), B.DTYPE[BF16], rows, c, ptr(res), B.DTYPE[torch.float32],
                                   B._Norm(post, ptr(w) if post else None, None), ptr(gate), rows, 0.5,
                                   B._Norm(pre, ptr(w) if pre else None, None), 1e-5, ptr(h), ptr(y), stream)
        assert st == 0
        assert torch.equal(both[0], h) if y is None else torch.equal(both[1], y)
    # null descriptors are the identity, no gate and no residual
    h = torch.empty_like(x)
    assert L.gated_residual_norm(ptr(x), B.DTYPE[BF16], rows, c, None, B.DTYPE[BF16], None, None, 0, -2.0, None, 1e-5, ptr(h),
                                 None, stream) == 0
    assert torch.equal(h, (x.double() * -2.0).to(BF16))


def test_attention_without_lse_is_the_same():
    g = gen(4)
    q, k, v = (torch.randn((200, h, 64), generator=g, device="cuda").to(BF16) for h in (4, 2, 2))
    a, none = spa.attention_prefill(q, k, v, offsets([200]))
    b, _ = spa.attention_prefill(q, k, v, offsets([200]), want_lse=True)
    assert none is None and torch.equal(a, b)


def test_broadcast_heads_and_rows():
    # strides of 0: one head's vectors for all, one row for all
    g = gen(5)
    q = torch.randn((70, 4, 64), generator=g, device="cuda").to(F16)
    k, v = (torch.randn((70, 1, 64), generator=g, device="cuda").to(F16) for _ in range(2))
    a = spa.attention_prefill(q, k.expand(-1, 2, -1), v.expand(-1, 2, -1), offsets([70]))[0]
    assert torch.equal(a, spa.attention_prefill(q, k, v, offsets([70]))[0])
    one = spa.attention_prefill(q[:1].expand(70, -1, -1), k, v, offsets([70]), causal=False)[0]
    assert torch.equal(one, one[:1].expand_as(one))
