"""The norm and rotation of queries and keys above 768 rows, where a workgroup takes two tokens, or several rows of two side by
side where the heads are few: without a cache, in place in a packed projection, and into each cache for every norm.  A row's
results are those of calls of few rows, bit for bit, and lie within the bounds of tests/test_rope_gpu.py."""
import pytest
import torch

import test_rope_gpu as T

pytestmark = pytest.mark.gpu

spa = pytest.importorskip("activation_sparsification_amd")

BF16, F16, I32 = torch.bfloat16, torch.float16, torch.int32
HEADS = [(32, 8, 128, 128, False), (40, 8, 64, 64, True), (1, 1, 8, 8, False), (3, 1, 32, 16, True), (1, 1, 32, 32, False), (2, 1, 256, 64, True),
         (5, 3, 96, 48, False)]


@pytest.fixture(scope="module")
def dev():
    assert torch.cuda.is_available(), "GPU tests need a device"
    return torch.device("cuda:0")


def arguments(norm, w, b, neighbours):
    args = dict(norm=norm, interleaved=neighbours)
    if norm != "none":
        args.update(q_weight=w[0], k_weight=w[1])
    if norm == "layer":
        args.update(q_bias=b[0], k_bias=b[1])
    return args


@pytest.mark.parametrize("t", [769, 1000, 2051])
@pytest.mark.parametrize("norm", ["none", "rms", "layer"])
@pytest.mark.parametrize("hq,hkv,d,rot,neighbours", HEADS)
def test_without_a_cache_and_in_place(dev, t, norm, hq, hkv, d, rot, neighbours):
    dtype = BF16 if t != 1000 else F16
    q, k, v, w, b = T.inputs(dev, t + d, t, hq, hkv, d, dtype)
    pos = torch.randint(0, 10 ** 6, (t,), generator=T.gen(dev, t), device=dev).to(I32)
    freq = T.frequencies(rot, dev)
    args = arguments(norm, w, b, neighbours)
    qo, ko = spa.qk_norm_rope(q, k, pos, freq, **args)
    for at in range(0, t, 500):
        s = slice(at, at + 500)
        qs, ks = spa.qk_norm_rope(q[s], k[s], pos[s], freq, **args)
        assert torch.equal(qo[s], qs) and torch.equal(ko[s], ks)
    bias = b if norm == "layer" else [None, None]
    weight = w if norm != "none" else [None, None]
    T.check(qo, T.reference(q, pos, freq, norm, weight[0], bias[0], 1e-5, neighbours), dtype)
    T.check(ko, T.reference(k, pos, freq, norm, weight[1], bias[1], 1e-5, neighbours), dtype)
    packed = torch.cat([q, k, v], dim=1)
    rest = packed[:, hq + hkv:].clone()
    spa.qk_norm_rope(packed[:, :hq], packed[:, hq:hq + hkv], pos, freq, q_out=packed[:, :hq], k_out=packed[:, hq:hq + hkv], **args)
    assert torch.equal(packed[:, :hq], qo) and torch.equal(packed[:, hq:hq + hkv], ko) and torch.equal(packed[:, hq + hkv:], rest)


@pytest.mark.parametrize("t", [769, 2051])
@pytest.mark.parametrize("norm", ["none", "rms"])
@pytest.mark.parametrize("hq,hkv,d,rot,neighbours", HEADS)
def test_into_the_cache_in_place(dev, t, norm, hq, hkv, d, rot, neighbours):
    q, k, v, w, b = T.inputs(dev, t + d, t, hq, hkv, d, BF16)
    g = T.gen(dev, t)
    pos = torch.randint(0, 10 ** 6, (t,), generator=g, device=dev).to(I32)
    freq = T.frequencies(rot, dev)
    slots = torch.randperm(t + 64, generator=g, device=dev)[:t].to(I32)
    slots[torch.rand(t, generator=g, device=dev) < 0.1] = -1
    n_pages = -(-(t + 64) // 16)
    args = arguments(norm, w, b, neighbours)
    qo, ko = spa.qk_norm_rope(q, k, pos, freq, **args)
    for fmt in T.FORMATS:
        one, other = (spa.new_kv_cache(n_pages, 16, hkv, d, BF16, fmt, dev) for _ in range(2))
        spa.kv_write(ko, v, slots, one)
        packed = torch.cat([q, k, v], dim=1)
        spa.qk_norm_rope(packed[:, :hq], packed[:, hq:hq + hkv], pos, freq, q_out=packed[:, :hq], k_out=packed[:, hq:hq + hkv],
                         v=packed[:, hq + hkv:], slots=slots, cache=other, **args)
        assert torch.equal(packed[:, :hq], qo) and torch.equal(packed[:, hq:hq + hkv], ko) and torch.equal(packed[:, hq + hkv:], v)
        for x, y in ((one.k, other.k), (one.v, other.v), (one.k_scale, other.k_scale), (one.v_scale, other.v_scale)):
            assert x is None or torch.equal(x.view(torch.uint8), y.view(torch.uint8))
