"""The cache, attention and norm calls beside autograd: they have no backward, and say so."""
import pytest
import torch

pytestmark = pytest.mark.gpu

spa = pytest.importorskip("activation_sparsification_amd")

BF16, I32 = torch.bfloat16, torch.int32


def arguments():
    """Every call, and the float tensors it takes (to be replaced one at a time)."""
    g = torch.Generator(device="cuda").manual_seed(5)
    rand = lambda *shape: torch.randn(shape, generator=g, device="cuda").to(BF16)
    cu, table = torch.tensor([0, 6], dtype=I32, device="cuda"), torch.tensor([[1, 0]], dtype=I32, device="cuda")
    slots, ln = torch.arange(16, 22, dtype=I32, device="cuda"), torch.tensor([6], dtype=I32, device="cuda")
    pages = dict(ck=torch.zeros((2, 2, 16, 64), dtype=BF16, device="cuda"), cv=torch.zeros((2, 2, 16, 64), dtype=BF16, device="cuda"))
    qkv = dict(q=rand(6, 4, 64), k=rand(6, 2, 64), v=rand(6, 2, 64))
    norm = dict(x=rand(5, 64), r=rand(5, 64), pw=rand(64), pb=rand(64), gate=rand(64), nw=rand(64), nb=rand(64))
    return {
        "prefill": (lambda q, k, v: spa.attention_prefill(q, k, v, cu)[0], qkv),
        "write": (lambda k, v, ck, cv: (spa.kv_write(k, v, slots, spa.KvCache(ck, cv)), ck)[1],
                  dict(k=qkv["k"], v=qkv["v"], **pages)),
        "read": (lambda ck, cv: spa.kv_read(spa.KvCache(ck, cv), table, cu, 6)[0], pages),
        "decode": (lambda q, ck, cv: spa.attention_decode(q, spa.KvCache(ck, cv), table, ln)[0], dict(q=qkv["q"][:1], **pages)),
        "norm": (lambda x, r, pw, pb, gate, nw, nb: spa.gated_residual_norm(x, r, post="layer", post_weight=pw, post_bias=pb,
                                                                          gate=gate, pre_weight=nw, pre_bias=nb)[1], norm),
    }


@pytest.mark.parametrize("name", ["prefill", "write", "read", "decode", "norm"])
def test_tensors_that_require_a_gradient_are_refused(name):
    call, given = arguments()[name]
    want = call(**given).clone()
    for which in given:
        now = dict(given)
        now[which] = given[which].clone().requires_grad_()
        with pytest.raises(ValueError, match="gradient"):
            call(**now)
        with torch.no_grad():
            assert torch.equal(call(**now), want)
        now[which] = (given[which].clone().requires_grad_() * 1)        # not a leaf
        with pytest.raises(ValueError, match="gradient"):
            call(**now)
        now[which] = now[which].detach()
        assert torch.equal(call(**now), want)


def test_outputs_that_require_a_gradient_are_refused():
    call, given = arguments()["prefill"]
    out = torch.empty((6, 4, 64), dtype=BF16, device="cuda", requires_grad=True)
    cu = torch.tensor([0, 6], dtype=I32, device="cuda")
    with pytest.raises(ValueError, match="gradient"):
        spa.attention_prefill(given["q"], given["k"], given["v"], cu, out=out)
    with torch.no_grad():
        assert spa.attention_prefill(given["q"], given["k"], given["v"], cu, out=out)[0] is out


def saved(t):
    """A loss whose backward needs the present values of t (which shares memory with what is returned)."""
    leaf = torch.ones_like(t, requires_grad=True)
    return (leaf * t).sum()


def test_writes_are_known_to_autograd():
    # a backward that kept the values a call has since overwritten is an error, not a wrong gradient
    all_calls = arguments()
    (_, a), (_, p), (_, n) = all_calls["prefill"], all_calls["decode"], all_calls["norm"]
    cu, table = torch.tensor([0, 6], dtype=I32, device="cuda"), torch.tensor([[1, 0]], dtype=I32, device="cuda")
    slots, ln = torch.arange(16, 22, dtype=I32, device="cuda"), torch.tensor([6], dtype=I32, device="cuda")
    cache = spa.new_kv_cache(2, 16, 2, 64, BF16, "int8")
    native = spa.KvCache(p["ck"], p["cv"])
    out, one = torch.zeros((6, 4, 64), dtype=BF16, device="cuda"), torch.zeros((1, 4, 64), dtype=BF16, device="cuda")
    k, v = torch.zeros_like(a["k"]), torch.zeros_like(a["v"])
    for name, targets, call in (
            ("prefill", [out], lambda: spa.attention_prefill(a["q"], a["k"], a["v"], cu, out=out)),
            ("decode", [one], lambda: spa.attention_decode(a["q"][:1], native, table, ln, out=one)),
            ("write", [native.k, native.v], lambda: spa.kv_write(a["k"], a["v"], slots, native)),
            ("write int8", [cache.k_scale, cache.v_scale], lambda: spa.kv_write(a["k"], a["v"], slots, cache)),
            ("read", [k, v], lambda: spa.kv_read(native, table, cu, 6, k_out=k, v_out=v)),
            ("norm", [n["r"], n["x"]], lambda: spa.gated_residual_norm(n["x"], n["r"], h_out=n["r"], y_out=n["x"]))):
        losses = [saved(t) for t in targets]
        call()
        for loss in losses:
            with pytest.raises(RuntimeError, match="modified by an inplace operation"):
                loss.backward()
        call()
        for t in targets:
            saved(t).backward()


def test_inference_tensors_are_written():
    with torch.inference_mode():
        call, given = arguments()["norm"]
        want = spa.gated_residual_norm(given["x"], given["r"])
        h, y = torch.empty_like(given["r"]), torch.empty_like(given["x"])
    got = spa.gated_residual_norm(given["x"], given["r"], h_out=h, y_out=y)
    assert got[0] is h and torch.equal(h, want[0]) and torch.equal(y, want[1])
