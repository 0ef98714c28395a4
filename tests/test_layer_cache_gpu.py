"""A KvCache works on the memory its tensors have when a call is made."""
import pytest
import torch

pytestmark = pytest.mark.gpu

spa = pytest.importorskip("activation_sparsification_amd")

BF16 = torch.bfloat16
FORMATS = ["native", "fp8", "int8"]


def inputs(t=20, h=2, d=64):
    g = torch.Generator(device="cuda").manual_seed(7)
    k, v, q = (torch.randn((t, n, d), generator=g, device="cuda").to(BF16) for n in (h, h, 4))
    table = torch.tensor([[2, 0]], dtype=torch.int32, device="cuda")
    pos = torch.arange(t, device="cuda")
    slots = (table[0, pos // 16].long() * 16 + pos % 16).to(torch.int32)
    return q[:1], k, v, slots, table, torch.tensor([t], dtype=torch.int32, device="cuda")


def parts(cache):
    return [x for x in (cache.k, cache.v, cache.k_scale, cache.v_scale) if x is not None]


@pytest.mark.parametrize("fmt", FORMATS)
def test_tensors_given_other_memory(fmt):
    q, k, v, slots, table, ln = inputs()
    want = spa.new_kv_cache(4, 16, 2, 64, BF16, fmt)
    spa.kv_write(k, v, slots, want)
    want_out, _ = spa.attention_decode(q, want, table, ln)
    cache = spa.new_kv_cache(4, 16, 2, 64, BF16, fmt)
    old = [x.detach() for x in parts(cache)]                    # the first memory stays alive, and stays as it is
    for x in parts(cache):
        x.set_(torch.zeros_like(x))
    spa.kv_write(k, v, slots, cache)
    for x, y, z in zip(parts(cache), parts(want), old):
        assert torch.equal(x.view(torch.uint8), y.view(torch.uint8)), "the write went elsewhere"
        assert not z.view(torch.uint8).any(), "the memory given up was written"
    out, _ = spa.attention_decode(q, cache, table, ln)
    assert torch.equal(out, want_out)
    for x, y in zip(parts(cache), parts(want)):
        x.set_(y.clone())
        y.zero_()
    out, _ = spa.attention_decode(q, cache, table, ln)
    assert torch.equal(out, want_out)
    got = spa.kv_read(cache, table, torch.tensor([0, 20], dtype=torch.int32, device="cuda"), 20, dtype=BF16)
    assert (got[0].float() - k.float()).abs().max() < 0.25 and (got[1].float() - v.float()).abs().max() < 0.25


@pytest.mark.parametrize("fmt", FORMATS)
def test_tensors_grown(fmt):
    # more pages: the calls and the sizes follow
    q, k, v, slots, table, ln = inputs()
    cache = spa.new_kv_cache(1, 16, 2, 64, BF16, fmt)
    old = [x.detach() for x in parts(cache)]
    for x in parts(cache):
        x.set_(torch.zeros((4, *x.shape[1:]), dtype=x.dtype, device=x.device))
    spa.kv_write(k, v, slots, cache)
    assert cache.n_pages == 4 and cache.page_size == 16 and cache.n_heads == 2 and cache.head_dim == 64
    got = spa.kv_read(cache, table, torch.tensor([0, 20], dtype=torch.int32, device="cuda"), 20, dtype=BF16)
    assert (got[0].float() - k.float()).abs().max() < 0.25 and (got[1].float() - v.float()).abs().max() < 0.25
    want = spa.new_kv_cache(4, 16, 2, 64, BF16, fmt)
    spa.kv_write(k, v, slots, want)
    assert torch.equal(spa.attention_decode(q, cache, table, ln)[0], spa.attention_decode(q, want, table, ln)[0])
    assert not any(x.view(torch.uint8).any() for x in old)


def refused(cache):
    q, k, v, slots, table, ln = inputs()
    for call in (lambda: spa.kv_write(k, v, slots, cache), lambda: spa.attention_decode(q, cache, table, ln),
                 lambda: spa.kv_read(cache, table, torch.tensor([0, 20], dtype=torch.int32, device="cuda"), 20, dtype=BF16)):
        with pytest.raises(ValueError):
            call()


@pytest.mark.parametrize("fmt", FORMATS)
def test_tensors_that_no_longer_fit_are_refused(fmt):
    def fresh():
        return spa.new_kv_cache(4, 16, 2, 64, BF16, fmt)

    cache = fresh()
    cache.v.set_(torch.zeros((3, 2, 16, 64), dtype=cache.v.dtype, device="cuda"))           # fewer pages than k
    refused(cache)
    cache = fresh()
    cache.k.untyped_storage().resize_(0)                                                    # its memory given back
    refused(cache)
    cache = fresh()
    cache.v.untyped_storage().resize_(cache.v.numel() * cache.v.element_size() // 2)
    refused(cache)
    cache = fresh()
    cache.k.transpose_(1, 2)                                                                # another layout
    refused(cache)
    if fmt != "native":
        cache = fresh()
        cache.v_scale.set_(torch.zeros((4, 2, 15), device="cuda"))
        refused(cache)
        cache = fresh()
        cache.k_scale.untyped_storage().resize_(0)
        refused(cache)


def test_other_tensors_without_their_memory_are_refused():
    q, k, v, slots, table, ln = inputs()
    cache = spa.new_kv_cache(4, 16, 2, 64, BF16)
    cu = torch.tensor([0, 1], dtype=torch.int32, device="cuda")
    x, w = torch.zeros((3, 64), dtype=BF16, device="cuda"), torch.zeros(64, dtype=BF16, device="cuda")
    for name, call in (("k", lambda t: spa.kv_write(t, v, slots, cache)), ("slots", lambda t: spa.kv_write(k, v, t, cache)),
                       ("q", lambda t: spa.attention_decode(t, cache, table, ln)),
                       ("table", lambda t: spa.attention_decode(q, cache, t, ln)),
                       ("kp", lambda t: spa.attention_prefill(q, t, v[:1], cu)), ("x", lambda t: spa.gated_residual_norm(t)),
                       ("w", lambda t: spa.gated_residual_norm(x, post="rms", post_weight=t)),
                       ("x", lambda t: spa.gated_residual_norm(x, t)), ("x", lambda t: spa.gated_residual_norm(x, h_out=t))):
        t = {"k": k, "slots": slots, "q": q, "table": table, "kp": k[:1], "x": x, "w": w}[name].clone()
        t.untyped_storage().resize_(t.numel() * t.element_size() - 1)
        with pytest.raises(ValueError, match="storage"):
            call(t)
