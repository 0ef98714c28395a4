"""The cache, attention and norm entry points on the host (CPU only, no device call): argument checks under
sanitizers, rejections through the C ABI before any launch, and the binding's surface."""
import ctypes
import inspect
import math
import os
import shutil
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
OK, INVALID, UNSUPPORTED = 0, 1, 2


def test_checks_under_sanitizers(tmp_path):
    cxx = shutil.which("g++")
    if cxx is None:
        pytest.skip("no host C++ compiler")
    exe = str(tmp_path / "layer_check_driver")
    cmd = [cxx, "-std=c++17", "-O1", "-g", "-fsanitize=address,undefined", "-fno-sanitize-recover=undefined", "-Wall",
           "-I", os.path.join(ROOT, "include"), "-I", os.path.join(ROOT, "activation_sparsification_amd", "csrc"),
           os.path.join(HERE, "native", "layer_check_driver.cpp"), "-o", exe]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0 and "sanitizer" in r.stderr.lower():
        pytest.skip("no sanitizer runtime for the host compiler")
    assert r.returncode == 0, r.stderr
    r = subprocess.run([exe], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stdout + r.stderr
    words = r.stdout.split()
    assert words[0] == "ok", r.stdout
    assert all(int(w) > 10000 for w in words[4:]), r.stdout        # every check accepts, not only rejects


@pytest.fixture(scope="module")
def B():
    import activation_sparsification_amd._binding as b
    b.lib()
    return b


def heads(B, data=4096, row=512, head=64):
    return B._Heads(data, row, head)


def cache(B, dtype=2, fmt=0, pages=4, page=16, h=2, d=64, k=4096, v=8192, ks=None, vs=None):
    return B._KvCache(dtype, fmt, pages, page, h, d, k, v, ks, vs)


def test_cache_rejections(B):
    L = B.lib()
    x = heads(B)
    good = cache(B)
    assert L.spa_kv_write(x, x, 0, None, good, None) == OK                       # no tokens
    assert L.spa_kv_write(x, x, -1, 256, good, None) == INVALID
    assert L.spa_kv_write(x, x, 4, None, good, None) == INVALID                  # no slots
    assert L.spa_kv_write(heads(B, None), x, 4, 256, good, None) == INVALID
    assert L.spa_kv_write(heads(B, row=-8), x, 4, 256, good, None) == INVALID
    assert L.spa_kv_write(heads(B, row=(1 << 23) + 8), x, 4, 256, good, None) == INVALID
    assert L.spa_kv_write(heads(B, data=4104), x, 4, 256, good, None) == UNSUPPORTED      # off 16 bytes
    assert L.spa_kv_write(heads(B, row=516), x, 4, 256, good, None) == UNSUPPORTED
    for bad, want in ((cache(B, dtype=7), INVALID), (cache(B, fmt=3), INVALID), (cache(B, pages=0), INVALID),
                      (cache(B, page=0), INVALID), (cache(B, h=0), INVALID), (cache(B, k=None), INVALID),
                      (cache(B, fmt=1), INVALID), (cache(B, fmt=2, ks=256), INVALID), (cache(B, d=0), INVALID),
                      (cache(B, dtype=0), UNSUPPORTED), (cache(B, d=60), UNSUPPORTED), (cache(B, d=264), UNSUPPORTED),
                      (cache(B, pages=1 << 26, page=16), UNSUPPORTED)):
        assert L.spa_kv_write(x, x, 4, 256, bad, None) == want
        assert L.spa_kv_read(bad, 256, 1, 4, 512, 8, 4096, 8192, None) == want
    assert L.spa_kv_write(x, x, 1 << 26, 256, good, None) == UNSUPPORTED         # more vectors than a launch has places
    assert L.spa_kv_read(good, 256, 0, 4, 512, 8, 4096, 8192, None) == OK        # no sequences
    assert L.spa_kv_read(good, 256, 1, 4, 512, 0, None, None, None) == OK        # no rows
    assert L.spa_kv_read(good, None, 1, 4, 512, 8, 4096, 8192, None) == INVALID
    assert L.spa_kv_read(good, 256, 1, 0, 512, 8, 4096, 8192, None) == INVALID
    assert L.spa_kv_read(good, 256, 1, 4, 512, 8, 4096, 8200, None) == INVALID   # unaligned output


def test_attention_rejections(B):
    L = B.lib()
    q, kv = heads(B), heads(B, row=128)

    def decode(q=q, n=2, hq=8, c=None, table=256, pages=4, lens=512, scale=0.125, out=4096, ws=8192, nb=1 << 40):
        return L.attention_decode(q, n, hq, c or cache(B), table, pages, lens, scale, out, None, ws, nb, None)

    assert decode(n=0) == OK
    for kw in (dict(n=-1), dict(hq=7), dict(hq=0), dict(scale=0.0), dict(scale=-1.0), dict(scale=math.nan), dict(scale=math.inf),
               dict(table=None), dict(lens=None), dict(out=None), dict(out=4104), dict(ws=None), dict(nb=64), dict(ws=8200),
               dict(q=heads(B, None)), dict(pages=-1)):
        assert decode(**kw) == INVALID, kw
    for kw in (dict(c=cache(B, dtype=0)), dict(pages=1 << 26), dict(q=heads(B, row=516)), dict(n=1 << 20, hq=512)):
        assert decode(**kw) == UNSUPPORTED, kw

    def prefill(q=q, k=kv, v=kv, dtype=2, tq=8, tk=8, hq=8, hkv=2, d=64, cq=256, ck=512, n=1, scale=0.125, out=4096):
        return L.attention_prefill(q, k, v, dtype, tq, tk, hq, hkv, d, cq, ck, n, 1, scale, out, None, None, 0, None)

    assert prefill(tq=0) == OK and prefill(n=0) == OK
    for kw in (dict(dtype=5), dict(tq=-1), dict(tk=-1), dict(hq=7), dict(hkv=0), dict(d=0), dict(cq=None), dict(ck=None),
               dict(n=-1), dict(scale=0.0), dict(scale=math.nan), dict(out=None), dict(out=4100), dict(k=heads(B, None)),
               dict(v=heads(B, row=-8))):
        assert prefill(**kw) == INVALID, kw
    for kw in (dict(dtype=0), dict(d=60), dict(d=264), dict(q=heads(B, data=4100)), dict(k=heads(B, row=132)), dict(n=1 << 20, hq=16)):
        assert prefill(**kw) == UNSUPPORTED, kw
    # few rows over many keys are divided: a call without the workspace for it is refused
    assert L.spa_attention_prefill_workspace_bytes(16, 100000, 1, 8, 64) >= 8 * 16 * 8 * 64 * 4
    assert prefill(tq=16, tk=100000) == INVALID
    assert L.spa_attention_prefill_workspace_bytes(8192, 8192, 1, 32, 128) == 0
    assert L.spa_attention_prefill_workspace_bytes(16, 200, 1, 8, 64) == 0
    assert L.spa_attention_decode_workspace_bytes(0, 8, 2, 64) == 0
    assert L.spa_attention_decode_workspace_bytes(4, 7, 2, 64) == 0
    assert L.spa_attention_decode_workspace_bytes(4, 8, 2, 64) > 0


def test_prompt_keys_are_divided_where_it_pays(B):
    # the join costs more than it brings for short prompts that leave a unit one workgroup, less for long ones
    need = B.lib().spa_attention_prefill_workspace_bytes
    assert need(700, 700, 1, 32, 128) == 0
    assert need(1200, 1200, 4, 16, 128) == 0
    assert need(4000, 4000, 1, 8, 128) == 2 * 4000 * 8 * (128 * 4 + 8)
    assert need(0, 0, 0, 8, 64) == 0


def test_norm_rejections(B):
    L = B.lib()

    def norm(x=4096, dtype=2, t=4, c=64, res=8192, st=2, post=None, gate=None, rows=0, scale=1.0, pre=None, eps=1e-5, h=12288,
             y=16384):
        return L.gated_residual_norm(x, dtype, t, c, res, st, post, gate, rows, scale, pre, eps, h, y, None)

    rms, bad = B._Norm(1, None, None), B._Norm(4, None, None)
    assert norm(t=0) == OK
    for kw in (dict(dtype=3), dict(st=-1), dict(t=-1), dict(c=0), dict(post=bad), dict(pre=bad), dict(eps=-1.0), dict(eps=math.nan),
               dict(scale=math.nan), dict(scale=math.inf), dict(gate=4096, rows=3), dict(gate=4096, rows=0), dict(rows=1),
               dict(x=None), dict(h=None, y=None), dict(h=4096, y=4096), dict(x=4104), dict(h=12290), dict(post=B._Norm(1, 4100, None))):
        assert norm(**kw) == INVALID, kw
    for kw in (dict(dtype=0, st=2), dict(dtype=1, st=2), dict(c=65537, pre=rms)):
        assert norm(**kw) == UNSUPPORTED, kw


def test_binding_surface():
    import activation_sparsification_amd as spa
    for name in ("KvCache", "attention_decode", "attention_prefill", "gated_residual_norm", "kv_read", "kv_write", "new_kv_cache"):
        assert name in dir(spa) and getattr(spa, name).__doc__
    assert list(inspect.signature(spa.attention_decode).parameters) == ["q", "cache", "page_table", "seq_lens", "scale",
                                                                        "want_lse", "out", "ws"]
    with pytest.raises(AttributeError):
        spa.no_such_name
    with pytest.raises(TypeError, match="missing required argument: 'slots'"):
        spa.kv_write(1, 2)
    with pytest.raises(TypeError, match="unexpected keyword argument 'mask'"):
        spa.attention_decode(1, 2, 3, 4, mask=5)
    with pytest.raises(TypeError, match="multiple values for argument 'q'"):
        spa.attention_prefill(1, 2, 3, 4, q=5)
    with pytest.raises(TypeError, match="expected a tensor"):
        spa.attention_prefill(1, 2, 3, 4)
    with pytest.raises(TypeError, match="at most 2 positional"):
        spa.gated_residual_norm(1, 2, 3)
    with pytest.raises(TypeError, match="expected a KvCache"):
        import torch
        spa.attention_decode(torch.zeros(1, 1, 8), "cache", 3, 4)
    with pytest.raises(ValueError, match="expected device tensors"):
        spa.new_kv_cache(1, 1, 1, 8, torch.bfloat16, device="cpu")
    with pytest.raises(ValueError, match="unknown format"):
        spa.new_kv_cache(1, 1, 1, 8, torch.bfloat16, "fp4", device="cpu")
    assert ctypes.sizeof(spa._binding._KvCache) == 6 * 4 + 4 * 8
