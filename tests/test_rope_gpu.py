"""The norm of queries and keys with the rotation by position on the GPU, against the formulas in 64 bits.

With u the unit roundoff of the 16-bit type, an output is off by at most
* u |y| for its rounding, no less than half the last place of a subnormal;
* 2^-17 of the size of the terms of its two normed elements, as for the other norms (tests/layer_ref.py);
* delta (|u_a| + |u_b|) for the angle: 3 float64 roundings of position * inv_freq / 2 pi, at most 2^-51 of the angle; the
  float32 rounding of the rest, below half a turn (2^-24 of pi: 2^-22), and of sine and cosine (2^-22 together).
"""
import math

import pytest
import torch

import layer_ref as R

pytestmark = pytest.mark.gpu

spa = pytest.importorskip("activation_sparsification_amd")

BF16, F16, I32 = torch.bfloat16, torch.float16, torch.int32
TINY = {BF16: 2.0 ** -134, F16: 2.0 ** -25}
FORMATS = ["native", "fp8", "int8", "mxfp4"]


@pytest.fixture(scope="module")
def dev():
    assert torch.cuda.is_available(), "GPU tests need a device"
    return torch.device("cuda:0")


def gen(dev, seed):
    return torch.Generator(device=dev).manual_seed(seed)


def frequencies(rot, dev, base=10000.0):
    half = rot // 2
    return (base ** (-torch.arange(half, device=dev, dtype=torch.float64) / max(half, 1))).float()


def reference(x, pos, freq, kind, w, b, eps, neighbours):
    """y and its bound without the output's own rounding, [t, heads, d] float64."""
    u, size = R.norm(x.double(), kind, w, b, eps)
    y, bound = u.clone(), 2.0 ** -17 * size
    if kind == "none":
        bound = torch.zeros_like(u)
    half = 0 if freq is None else len(freq)
    if half:
        i = torch.arange(half, device=x.device)
        a, c = (2 * i, 2 * i + 1) if neighbours else (i, i + half)
        angle = pos.double()[:, None] * freq.double()
        cos, sin = angle.cos()[:, None], angle.sin()[:, None]
        y[..., a], y[..., c] = u[..., a] * cos - u[..., c] * sin, u[..., a] * sin + u[..., c] * cos
        delta = 2.0 ** -21 + 2.0 ** -51 * angle.abs()[:, None]
        turn = delta * (u[..., a].abs() + u[..., c].abs())
        ba, bc = bound[..., a], bound[..., c]
        bound[..., a] = ba * cos.abs() + bc * sin.abs() + turn
        bound[..., c] = ba * sin.abs() + bc * cos.abs() + turn
    return y, bound


def check(got, ref, dtype):
    y, bound = ref
    u = R.U[dtype]
    err = (got.double() - y).abs()
    limit = (torch.maximum(u * y.abs(), torch.full_like(y, TINY[dtype])) + bound) * (1 + u)
    assert torch.isfinite(got).all()
    assert (err <= limit).all(), f"error {(err / limit).max().item():.3f} of its bound"


def inputs(dev, seed, t, hq, hkv, d, dtype, weights=True):
    g = gen(dev, seed)
    x = (torch.randn((t, hq + 2 * hkv, d), generator=g, device=dev) * 1.5 + 0.1).to(dtype)
    w = [(1 + 0.3 * torch.randn(d, generator=g, device=dev)).to(dtype) for _ in range(2)] if weights else [None, None]
    b = [(0.2 * torch.randn(d, generator=g, device=dev)).to(dtype) for _ in range(2)] if weights else [None, None]
    return x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:], w, b


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("norm", ["none", "rms", "layer"])
@pytest.mark.parametrize("neighbours", [False, True])
@pytest.mark.parametrize("t,hq,hkv,d,rot", [(1, 1, 1, 8, 8), (3, 4, 2, 64, 64), (5, 32, 8, 128, 128), (17, 3, 1, 96, 48),
                                            (300, 7, 3, 64, 16), (261, 2, 2, 256, 256), (2, 5, 5, 40, 24), (9, 2, 1, 80, 80),
                                            (4, 40, 1, 32, 32), (700, 1, 1, 128, 64)])
def test_shapes(dev, dtype, norm, neighbours, t, hq, hkv, d, rot):
    q, k, _, w, b = inputs(dev, t + d, t, hq, hkv, d, dtype)
    pos = torch.randint(0, 5000, (t,), generator=gen(dev, 1), device=dev).to(I32)
    freq = frequencies(rot, dev)
    args = dict(norm=norm, q_weight=w[0], k_weight=w[1], eps=1e-6, interleaved=neighbours)
    if norm == "layer":
        args.update(q_bias=b[0], k_bias=b[1])
    qo, ko = spa.qk_norm_rope(q, k, pos, freq, **args)
    for got, x, i in ((qo, q, 0), (ko, k, 1)):
        check(got, reference(x, pos, freq, norm, w[i], b[i] if norm == "layer" else None, 1e-6, neighbours), dtype)


@pytest.mark.parametrize("dtype", [BF16, F16])
def test_far_positions(dev, dtype):
    # positions up to the end of their type, negative ones, frequencies of one and tiny ones
    q, k, _, _, _ = inputs(dev, 7, 12, 4, 2, 128, dtype)
    pos = torch.tensor([0, 1, -1, 4095, 131071, 1000003, 2 ** 24 + 1, 2 ** 30 + 7, 2 ** 31 - 1, -2 ** 31, -77777, 5], dtype=I32, device=dev)
    for base in (10000.0, 500000.0, 1.0):
        freq = frequencies(128, dev, base)
        for neighbours in (False, True):
            qo, ko = spa.qk_norm_rope(q, k, pos, freq, norm="none", interleaved=neighbours)
            check(qo, reference(q, pos, freq, "none", None, None, 0.0, neighbours), dtype)
            check(ko, reference(k, pos, freq, "none", None, None, 0.0, neighbours), dtype)


def test_without_rotation_or_weights(dev):
    q, k, _, w, b = inputs(dev, 3, 33, 4, 2, 64, BF16)
    qo, ko = spa.qk_norm_rope(q, k, norm="none")
    assert torch.equal(qo, q) and torch.equal(ko, k)                        # a copy
    qo, ko = spa.qk_norm_rope(q, k)                                         # rms without weights
    check(qo, reference(q, None, None, "rms", None, None, 1e-5, False), BF16)
    empty = torch.empty(0, device=dev)
    again, _ = spa.qk_norm_rope(q, k, torch.zeros(33, dtype=I32, device=dev), empty)
    assert torch.equal(again, qo)
    qo, ko = spa.qk_norm_rope(q, k, norm="layer", q_weight=w[0], k_bias=b[1])       # a weight for one, a bias for the other
    check(qo, reference(q, None, None, "layer", w[0], None, 1e-5, False), BF16)
    check(ko, reference(k, None, None, "layer", None, b[1], 1e-5, False), BF16)


def test_position_zero_keeps_the_vector(dev):
    q, k, _, _, _ = inputs(dev, 5, 20, 2, 1, 128, F16)
    qo, ko = spa.qk_norm_rope(q, k, torch.zeros(20, dtype=I32, device=dev), frequencies(128, dev), norm="none")
    assert torch.equal(qo, q) and torch.equal(ko, k)


def test_small_and_large_heads(dev):
    # zeros (the norm's eps decides), values whose squares leave 16 bits, tiny ones
    for dtype, big in ((BF16, 2.0 ** 60), (F16, 60000.0)):
        x = torch.randn((6, 3, 64), generator=gen(dev, 2), device=dev)
        x[0] = 0.0
        x[1] = x[1].clamp(-1, 1) * big
        x[2] *= 1e-6
        x = x.to(dtype)
        for norm in ("rms", "layer"):
            qo, _ = spa.qk_norm_rope(x, x[:, :1], norm=norm, eps=1e-12)
            check(qo, reference(x, None, None, norm, None, None, 1e-12, False), dtype)
            assert (qo[0] == 0).all()


@pytest.mark.parametrize("neighbours", [False, True])
def test_in_place_and_strided_outputs(dev, neighbours):
    q, k, v, w, _ = inputs(dev, 11, 130, 8, 2, 128, BF16)
    pos = torch.arange(130, dtype=I32, device=dev) + 77
    freq = frequencies(64, dev)
    args = dict(q_weight=w[0], k_weight=w[1], interleaved=neighbours)
    want = spa.qk_norm_rope(q, k, pos, freq, **args)
    x = torch.empty((130, 20, 128), dtype=BF16, device=dev).fill_(5.0)
    spread = x[:, 3:11], x[:, 12:14]
    got = spa.qk_norm_rope(q, k, pos, freq, q_out=spread[0], k_out=spread[1], **args)
    assert got[0] is spread[0] and got[1] is spread[1]
    assert torch.equal(spread[0], want[0]) and torch.equal(spread[1], want[1])
    assert (x[:, :3] == 5).all() and (x[:, 11] == 5).all() and (x[:, 14:] == 5).all()
    flipped = torch.empty((8, 130, 128), dtype=BF16, device=dev).transpose(0, 1)        # heads outermost
    spa.qk_norm_rope(q, k, pos, freq, q_out=flipped, **args)
    assert torch.equal(flipped, want[0])
    whole = torch.cat([q, k, v], dim=1)
    rest = whole[:, 10:].clone()
    spa.qk_norm_rope(whole[:, :8], whole[:, 8:10], pos, freq, q_out=whole[:, :8], k_out=whole[:, 8:10], **args)
    assert torch.equal(whole[:, :8], want[0]) and torch.equal(whole[:, 8:10], want[1]) and torch.equal(whole[:, 10:], rest)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("t,hq,hkv,d,rot,page,neighbours", [(1, 4, 1, 128, 128, 16, False), (48, 32, 8, 128, 128, 16, False), (300, 6, 3, 64, 32, 7, True),
                                                            (37, 2, 2, 96, 96, 1, False), (33, 3, 1, 40, 8, 100, False), (270, 2, 1, 256, 64, 32, True),
                                                            (20, 1, 1, 8, 8, 5, True)])
def test_cache_as_written_apart(dev, fmt, dtype, t, hq, hkv, d, rot, page, neighbours):
    q, k, v, w, b = inputs(dev, t + d, t, hq, hkv, d, dtype)
    g = gen(dev, t)
    pos = torch.randint(0, 100000, (t,), generator=g, device=dev).to(I32)
    freq = frequencies(rot, dev)
    n_pages = -(-t // page) + 2
    slots = torch.randperm(n_pages * page, generator=g, device=dev)[:t].to(I32)
    slots[torch.rand(t, generator=g, device=dev) < 0.1] = -1
    if t > 10:
        slots[3], slots[7] = n_pages * page, 2 ** 31 - 1
    caches = [spa.new_kv_cache(n_pages, page, hkv, d, dtype, fmt, dev) for _ in range(3)]
    parts = [[x for x in (c.k, c.v, c.k_scale, c.v_scale) if x is not None] for c in caches]
    for c in parts:
        for x in c:
            x.view(torch.uint8).fill_(0x35)
    args = dict(norm="layer", q_weight=w[0], k_weight=w[1], q_bias=b[0], k_bias=b[1], interleaved=neighbours)
    qw, kw = spa.qk_norm_rope(q, k, pos, freq, **args)
    spa.kv_write(kw, v, slots, caches[0])
    qo, ko = spa.qk_norm_rope(q, k, pos, freq, v=v, slots=slots, cache=caches[1], **args)
    assert ko is None and torch.equal(qo, qw)
    qo, ko = spa.qk_norm_rope(q, k, pos, freq, v=v, slots=slots, cache=caches[2], k_out=torch.empty_like(kw), **args)
    assert torch.equal(qo, qw) and torch.equal(ko, kw)
    for want, one, two in zip(*parts):
        assert torch.equal(want.view(torch.uint8), one.view(torch.uint8)) and torch.equal(want.view(torch.uint8), two.view(torch.uint8))


@pytest.mark.parametrize("t", [768, 769, 1000, 2051])
@pytest.mark.parametrize("hq,hkv,d,rot,neighbours", [(5, 3, 128, 64, False), (3, 1, 48, 48, True), (2, 2, 256, 256, False)])
def test_few_and_many_tokens_agree(dev, t, hq, hkv, d, rot, neighbours):
    # a row's outputs and cached vectors do not depend on how many rows the call has
    q, k, v, w, b = inputs(dev, t + d, t, hq, hkv, d, BF16)
    g = gen(dev, t)
    pos = torch.randint(0, 2 ** 31 - 1, (t,), generator=g, device=dev).to(I32)
    freq = frequencies(rot, dev)
    slots = torch.randperm(t + 64, generator=g, device=dev)[:t].to(I32)
    slots[torch.rand(t, generator=g, device=dev) < 0.1] = -1
    n_pages = -(-(t + 64) // 16)
    args = dict(q_weight=w[0], k_weight=w[1], q_bias=b[0], k_bias=b[1], norm="layer", interleaved=neighbours)
    for fmt in FORMATS:
        one, other = (spa.new_kv_cache(n_pages, 16, hkv, d, BF16, fmt, dev) for _ in range(2))
        qo, ko = spa.qk_norm_rope(q, k, pos, freq, v=v, slots=slots, cache=one, k_out=torch.empty(k.shape, dtype=BF16, device=dev), **args)
        for at in range(0, t, 500):
            s = slice(at, at + 500)
            qs, ks = spa.qk_norm_rope(q[s], k[s], pos[s], freq, v=v[s], slots=slots[s], cache=other,
                                      k_out=torch.empty(k[s].shape, dtype=BF16, device=dev), **args)
            assert torch.equal(qo[s], qs) and torch.equal(ko[s], ks)
        for x, y in ((one.k, other.k), (one.v, other.v), (one.k_scale, other.k_scale), (one.v_scale, other.v_scale)):
            assert x is None or torch.equal(x.view(torch.uint8), y.view(torch.uint8))
    check(qo, reference(q, pos, freq, "layer", w[0], b[0], 1e-5, neighbours), BF16)
    check(ko, reference(k, pos, freq, "layer", w[1], b[1], 1e-5, neighbours), BF16)


@pytest.mark.parametrize("fmt", FORMATS)
def test_nonfinite_heads_stay_by_themselves(dev, fmt):
    q, k, v, w, _ = inputs(dev, 1, 40, 4, 2, 128, BF16)
    pos, freq = torch.arange(40, dtype=I32, device=dev), frequencies(128, dev)
    slots = torch.arange(40, dtype=I32, device=dev)
    clean, dirty = (spa.new_kv_cache(3, 16, 2, 128, BF16, fmt, dev) for _ in range(2))
    want, _ = spa.qk_norm_rope(q, k, pos, freq, q_weight=w[0], v=v, slots=slots, cache=clean)
    q2, k2, v2 = q.clone(), k.clone(), v.clone()
    q2[5, 1, 0], q2[6, 3, 127], k2[9, 1, 64], v2[11, 0, 3] = math.nan, math.inf, -math.inf, math.nan
    got, _ = spa.qk_norm_rope(q2, k2, pos, freq, q_weight=w[0], v=v2, slots=slots, cache=dirty)
    hit = torch.zeros((40, 4), dtype=torch.bool, device=dev)
    hit[5, 1] = hit[6, 3] = True
    assert torch.isnan(got[hit]).any(-1).all() and torch.equal(got[~hit], want[~hit])
    table = torch.arange(3, dtype=I32, device=dev)[None]
    cu = torch.tensor([0, 40], dtype=I32, device=dev)
    a, b = (spa.kv_read(c, table, cu, 40, dtype=BF16) for c in (clean, dirty))
    for i, (row, head) in enumerate(((9, 1), (11, 0))):
        keep = torch.ones((40, 2), dtype=torch.bool, device=dev)
        keep[row, head] = False
        assert torch.equal(a[i][keep], b[i][keep]) and torch.isnan(b[i][row, head]).any()


def test_captured_calls_follow_later_positions(dev):
    q, k, v, w, _ = inputs(dev, 9, 24, 8, 2, 128, BF16)
    freq = frequencies(128, dev)
    pos, slots = torch.zeros(24, dtype=I32, device=dev), torch.full((24,), -1, dtype=I32, device=dev)
    cache, other = (spa.new_kv_cache(8, 16, 2, 128, BF16, "mxfp4", dev) for _ in range(2))
    out = torch.empty(q.shape, dtype=BF16, device=dev)

    def step(c, o):
        spa.qk_norm_rope(q, k, pos, freq, q_weight=w[0], k_weight=w[1], q_out=o, v=v, slots=slots, cache=c)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(cache, out)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(cache, out)
    for i in range(4):
        pos.copy_(torch.randint(0, 10 ** 6, (24,), dtype=I32))
        slots.copy_(torch.randperm(128, dtype=I32)[:24])
        graph.replay()
        torch.cuda.synchronize()
        want = torch.empty_like(out)
        step(other, want)
        assert torch.equal(out, want)
        for a, b in ((cache.k, other.k), (cache.v, other.v), (cache.k_scale, other.k_scale), (cache.v_scale, other.v_scale)):
            assert torch.equal(a, b)


def test_other_stream_and_many_rows(dev):
    # more rows than one launch dimension of small grids; queued behind its inputs on another stream
    t = 70000
    st = torch.cuda.Stream()
    with torch.cuda.stream(st):
        q, k, _, w, _ = inputs(dev, 2, t, 2, 1, 64, BF16)
        pos, freq = torch.arange(t, dtype=I32, device=dev), frequencies(64, dev)
        qo, ko = spa.qk_norm_rope(q, k, pos, freq, q_weight=w[0], k_weight=w[1])
    st.synchronize()
    check(qo, reference(q, pos, freq, "rms", w[0], None, 1e-5, False), BF16)
    check(ko, reference(k, pos, freq, "rms", w[1], None, 1e-5, False), BF16)


def test_no_rows(dev):
    x = torch.empty((0, 6, 64), dtype=BF16, device=dev)
    q, k = spa.qk_norm_rope(x[:, :4], x[:, 4:], torch.empty(0, dtype=I32, device=dev), frequencies(64, dev))
    assert q.shape == (0, 4, 64) and k.shape == (0, 2, 64)


def test_tensors_that_require_a_gradient_are_refused(dev):
    q, k, v, w, b = inputs(dev, 1, 6, 4, 2, 64, BF16)
    pos, freq, slots = torch.arange(6, dtype=I32, device=dev), frequencies(64, dev), torch.arange(6, dtype=I32, device=dev)
    cache = spa.new_kv_cache(1, 16, 2, 64, BF16, "native", dev)
    given = dict(q=q, k=k, inv_freq=freq, q_weight=w[0], k_weight=w[1], q_bias=b[0], k_bias=b[1], v=v, q_out=torch.empty_like(q),
                 k_out=torch.empty_like(k))
    spa.qk_norm_rope(positions=pos, slots=slots, cache=cache, norm="layer", **given)
    for name in given:
        now = dict(given)
        now[name] = given[name].clone().requires_grad_()
        with pytest.raises(ValueError, match="gradient"):
            spa.qk_norm_rope(positions=pos, slots=slots, cache=cache, norm="layer", **now)
        with torch.no_grad():
            spa.qk_norm_rope(positions=pos, slots=slots, cache=cache, norm="layer", **now)
    leaf = torch.ones_like(cache.k, requires_grad=True)
    loss = (leaf * cache.k).sum()
    spa.qk_norm_rope(positions=pos, slots=slots, cache=cache, norm="layer", **given)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        loss.backward()


def test_binding_refusals(dev):
    q, k, v, w, _ = inputs(dev, 1, 6, 4, 2, 64, BF16)
    pos, freq, slots = torch.arange(6, dtype=I32, device=dev), frequencies(64, dev), torch.arange(6, dtype=I32, device=dev)
    cache = spa.new_kv_cache(1, 16, 2, 64, BF16, "native", dev)
    for kw, match in ((dict(positions=pos), "belong together"), (dict(inv_freq=freq), "belong together"),
                      (dict(positions=pos[:5], inv_freq=freq), "positions"), (dict(positions=pos.long(), inv_freq=freq), "positions"),
                      (dict(positions=pos, inv_freq=freq.double()), "inv_freq"), (dict(positions=pos, inv_freq=torch.ones(33, device=dev)), "more pairs"),
                      (dict(norm="batch"), "unknown norm"), (dict(q_weight=w[0].float()), "q_norm"), (dict(k_weight=w[1][:32]), "k_norm"),
                      (dict(q_out=torch.empty_like(k)), "q_out"), (dict(k_out=k.float()), "k_out"), (dict(v=v), "belong together"),
                      (dict(slots=slots), "belong together"), (dict(cache=cache), "belong together"),
                      (dict(v=v, slots=slots[:3], cache=cache), "slots"), (dict(v=v[:, :1], slots=slots, cache=cache), "v: differs"),
                      (dict(v=v, slots=slots, cache=spa.new_kv_cache(1, 16, 2, 64, F16, "native", dev)), "pages"),
                      (dict(v=v, slots=slots, cache=spa.new_kv_cache(1, 16, 4, 64, BF16, "native", dev)), "other heads")):
        with pytest.raises(ValueError, match=match):
            spa.qk_norm_rope(q, k, **kw)
    with pytest.raises(ValueError, match="both the same"):
        spa.qk_norm_rope(q, k.to(F16))
    with pytest.raises(ValueError, match="rows or head_dim"):
        spa.qk_norm_rope(q, k[:5])
    with pytest.raises(spa.SpaError):                                       # overlapping outputs
        spa.qk_norm_rope(q, k, q_out=torch.empty((6, 1, 64), dtype=BF16, device=dev).expand(6, 4, 64))
    with pytest.raises(spa.SpaError):                                       # pairs that lanes do not hold
        spa.qk_norm_rope(q, k, pos, frequencies(12, dev))
    with pytest.raises(spa.SpaError):
        spa.qk_norm_rope(q.float(), k.float())
