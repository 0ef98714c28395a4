"""The 4-bit cache on the host (CPU only): refusals through the C ABI before any launch, the binding's checks, and the
format's own properties in the reference."""
import pytest
import torch

import mxfp4_ref as M

OK, INVALID, UNSUPPORTED = 0, 1, 2


@pytest.fixture(scope="module")
def B():
    import activation_sparsification_amd._binding as b
    b.lib()
    return b


def cache(B, dtype=2, pages=4, page=16, h=2, d=64, k=4096, v=8192, ks=12288, vs=16384):
    return B._KvCache(dtype, 3, pages, page, h, d, k, v, ks, vs)


def test_refusals(B):
    L = B.lib()
    x, q = B._Heads(4096, 512, 64), B._Heads(4096, 1024, 64)
    assert L.spa_kv_write(x, x, 0, None, cache(B), None) == OK
    for bad, want in ((cache(B, dtype=9), INVALID), (cache(B, ks=None), INVALID), (cache(B, vs=None), INVALID),
                      (cache(B, ks=12290), INVALID), (cache(B, vs=16392), INVALID), (cache(B, k=4104), INVALID), (cache(B, page=0), INVALID),
                      (cache(B, d=0), INVALID), (cache(B, dtype=0), UNSUPPORTED), (cache(B, d=36), UNSUPPORTED),
                      (cache(B, d=264), UNSUPPORTED), (cache(B, pages=1 << 26), UNSUPPORTED)):
        assert L.spa_kv_write(x, x, 4, 256, bad, None) == want
        assert L.spa_kv_read(bad, 256, 1, 4, 512, 8, 4096, 8192, None) == want
        assert L.attention_decode(q, 2, 8, bad, 256, 4, 512, 0.125, 4096, None, 8192, 1 << 40, None) == want
    assert L.attention_decode(q, 2, 7, cache(B), 256, 4, 512, 0.125, 4096, None, 8192, 1 << 40, None) == INVALID
    assert L.attention_decode(q, 2, 8, cache(B), 256, 4, 512, 0.125, 4096, None, 8192, 64, None) == INVALID
    assert L.attention_decode(q, 0, 8, cache(B), 256, 4, 512, 0.125, 4096, None, 8192, 1 << 40, None) == OK
    assert L.spa_kv_write(x, x, 4, 256, B._KvCache(2, 4, 4, 16, 2, 64, 4096, 8192, 4096, 4096), None) == INVALID      # no such format


def test_binding_refusals():
    import activation_sparsification_amd as spa
    with pytest.raises(ValueError, match="expected device tensors"):
        spa.new_kv_cache(1, 1, 1, 8, torch.bfloat16, "mxfp4", device="cpu")
    with pytest.raises(ValueError, match="half a byte"):
        spa.new_kv_cache(1, 1, 1, 7, torch.bfloat16, "mxfp4", device="cpu")


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_reference_format(dtype):
    # every value that a code and a scale stand for is kept, unless it would carry a lower scale; nothing leaves the type
    g = torch.Generator().manual_seed(1)
    x = torch.randn((500, 64), generator=g) * torch.exp2(torch.randint(-12, 12, (500, 1), generator=g).float())
    x = x.to(dtype)
    codes, scales = M.quantise(x, dtype)
    held = M.values(M.pack(codes)[:, None, None], scales.to(torch.uint8)[:, None, :, None])[:, 0, 0]
    step = torch.exp2(scales.double() - 127).repeat_interleave(32, dim=-1)
    assert ((held - x.double()).abs() <= step).all()                    # half the step below the top code, or less
    again, same = M.quantise(held, dtype)
    keep = held.abs().view(500, 2, 32).amax(-1) > 3.5 * torch.exp2(scales.double() - 127)
    keep = keep.repeat_interleave(32, dim=-1)
    assert torch.equal(torch.where(keep, again, codes), codes)
    top = torch.full((1, 32), torch.finfo(dtype).max).to(dtype)
    c, s = M.quantise(top, dtype)
    assert M.values(M.pack(c)[:, None, None], s.to(torch.uint8)[:, None, :, None]).max() <= torch.finfo(dtype).max
