"""The calls around a server's cache on the host (CPU only): their argument checks swept under sanitizers, outputs that overlap,
the device that they launch on, and the binding's surface."""
import inspect
import os
import shutil
import subprocess
import sys
import sysconfig

import pytest
import torch

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
INVALID = 1


def test_checks_under_sanitizers(tmp_path):
    cxx = shutil.which("g++")
    if cxx is None:
        pytest.skip("no host C++ compiler")
    exe = str(tmp_path / "serving_check_driver")
    cmd = [cxx, "-std=c++17", "-O1", "-g", "-fsanitize=address,undefined", "-fno-sanitize-recover=undefined", "-Wall",
           "-I", os.path.join(ROOT, "include"), "-I", os.path.join(ROOT, "activation_sparsification_amd", "csrc"),
           os.path.join(HERE, "native", "serving_check_driver.cpp"), "-o", exe]
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


def test_plan_outputs_lie_apart(B):
    # refused before a launch: the calls below would have their GPU write one argument over another
    base = dict(lens=4096, fresh=8192, done=12288, table=16384, pages=20480, count=24576, count_out=28672, slots=32768, pos=36864,
                cq=40960, ck=45056, lo=49152)

    def call(**kw):
        a = {**base, **kw}
        return B.lib().spa_kv_plan(a["lens"], a["fresh"], a["done"], 8, a["table"], 4, 16, B._PagePool(a["pages"], a["count"], a["count_out"], 64), 32,
                                   a["slots"], a["pos"], a["cq"], a["ck"], a["lo"], None)

    for name in ("lens", "fresh", "done", "table", "pages", "count"):
        for out in ("count_out", "slots", "pos", "cq", "ck", "lo", "table", "pages"):
            if name == out or (name, out) in (("lens", "lo"), ("count", "count_out")):
                continue
            assert call(**{out: base[name]}) == INVALID, (name, out)
    assert call(lo=base["lens"] + 4) == INVALID and call(count_out=base["count"] - 4) == INVALID
    assert call(pos=base["slots"] + 124) == INVALID and call(ck=base["cq"] + 32) == INVALID


def test_rope_outputs_lie_apart(B):
    h = lambda data, row=1024, head=64: B._Heads(data, row, head)
    one, two, three = 65536, 131072, 262144

    def call(qo, ko, v=None, c=None, slots=None):
        return B.lib().qk_norm_rope(h(one), h(two), v, 2, 4, 8, 2, 64, 4096, B._Rope(4096, 64, 0), None, None, 1e-5, qo, ko, slots, c, None)

    for qo, ko in ((h(three), h(three)), (h(two), h(three)), (h(three), h(one)), (h(one, 2048), h(two)), (h(one), h(two, 1024, 128))):
        assert call(qo, ko) == INVALID
    c = B._KvCache(2, 0, 4, 16, 2, 64, 4096, 8192, None, None)
    assert call(h(one), h(three), v=h(three), c=c, slots=256) == INVALID
    assert call(h(three), None, v=h(three), c=c, slots=256) == INVALID


# The recorder takes the place of torch's device switch for good, so the calls have a process of their own.
PROGRAM = """
import sys
sys.path[:0] = [{build!r}, {root!r}]
import torch
import device_recorder as R
import activation_sparsification_amd as spa
R.install()
bf, i32, u8 = torch.bfloat16, torch.int32, torch.uint8
def f(*shape, dtype=bf): return R.fake(shape, dtype, 1)
q, kv, cu, ints = f(2, 4, 64), f(2, 2, 64), f(2, dtype=i32), f(2, dtype=i32)
four = spa.KvCache(f(2, 2, 16, 32, dtype=u8), f(2, 2, 16, 32, dtype=u8), f(2, 2, 2, 16, dtype=u8), f(2, 2, 2, 16, dtype=u8))
need = spa.lib().spa_attention_decode_workspace_bytes(2, 4, 2, 64)
ws = f(need, dtype=u8) if need <= 65536 else f(65536, dtype=u8)
calls = dict(
    kv_plan=lambda: spa.kv_plan(ints, ints, f(2, 3, dtype=i32), 16, f(8, dtype=i32), f(2, dtype=i32), 4, slots=f(4, dtype=i32),
                                positions=f(4, dtype=i32), cu_q=f(3, dtype=i32), cu_k=f(3, dtype=i32), lens_out=f(2, dtype=i32),
                                count_out=f(2, dtype=i32)),
    qk_norm_rope=lambda: spa.qk_norm_rope(q, kv, cu, f(32, dtype=torch.float32), q_out=q, k_out=kv),
    qk_norm_rope_cache=lambda: spa.qk_norm_rope(q, kv, cu, f(32, dtype=torch.float32), q_out=q, v=kv, slots=ints, cache=four),
    kv_write=lambda: spa.kv_write(kv, kv, ints, four),
    kv_read=lambda: spa.kv_read(four, f(1, 2, dtype=i32), cu, 2, k_out=kv, v_out=kv),
    attention_decode=lambda: spa.attention_decode(q, four, f(2, 2, dtype=i32), ints, out=q, ws=ws))
R.switches()
for name, call in calls.items():
    try:
        call()
        print(name, 'launched')
    except (RuntimeError, ValueError):
        print(name, *R.switches())
"""


def test_calls_switch_to_their_tensors_device(tmp_path):
    cxx = shutil.which("g++")
    if cxx is None:
        pytest.skip("no host C++ compiler")
    if torch.cuda.is_available():
        pytest.skip("for hosts without a GPU: nothing may be launched on tensors that are not there")
    t = os.path.dirname(torch.__file__)
    rocm = os.environ.get("ROCM_PATH", "/opt/rocm")
    cmd = [cxx, "-O0", "-std=c++17", "-fPIC", "-shared", "-D__HIP_PLATFORM_AMD__=1", "-DUSE_ROCM",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", "-isystem", os.path.join(t, "include"),
           "-isystem", os.path.join(t, "include/torch/csrc/api/include"), "-isystem", os.path.join(rocm, "include"),
           "-isystem", sysconfig.get_paths()["include"], os.path.join(HERE, "native", "device_recorder.cpp"), "-o",
           str(tmp_path / "device_recorder.so"), "-L", os.path.join(t, "lib"), "-ltorch_python", "-ltorch_cpu", "-lc10"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    r = subprocess.run([sys.executable, "-c", PROGRAM.format(build=str(tmp_path), root=ROOT)], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr
    got = {w[0]: w[1:] for w in (line.split() for line in r.stdout.splitlines()) if w}
    assert sorted(got) == ["attention_decode", "kv_plan", "kv_read", "kv_write", "qk_norm_rope", "qk_norm_rope_cache"], r.stdout
    for name, seen in got.items():
        assert seen == ["1", "0"], f"{name}: devices made current: {seen}"


def test_binding_surface():
    import activation_sparsification_amd as spa
    for name in ("kv_plan", "qk_norm_rope", "new_page_pool"):
        assert name in dir(spa) and getattr(spa, name).__doc__
    assert list(inspect.signature(spa.kv_plan).parameters) == ["lens", "new", "page_table", "page_size", "free_pages", "free_count", "t", "done",
                                                               "slots", "positions", "cu_q", "cu_k", "lens_out", "count_out"]
    assert list(inspect.signature(spa.qk_norm_rope).parameters) == ["q", "k", "positions", "inv_freq", "norm", "q_weight", "k_weight", "q_bias",
                                                                    "k_bias", "eps", "interleaved", "q_out", "k_out", "v", "slots", "cache"]
    with pytest.raises(TypeError, match="missing required argument: 't'"):
        spa.kv_plan(1, 2, 3, 4, 5, 6)
    with pytest.raises(TypeError, match="unexpected keyword argument 'mask'"):
        spa.qk_norm_rope(1, 2, mask=3)
    with pytest.raises(TypeError, match="positional"):
        spa.qk_norm_rope(1, 2, 3, 4, "rms")
    with pytest.raises(TypeError, match="expected a tensor"):
        spa.kv_plan(1, 2, 3, 4, 5, 6, 7)
    with pytest.raises(ValueError, match="device tensor"):
        x = torch.zeros(2, dtype=torch.int32)
        spa.kv_plan(x, x, x[None], 16, x, x, 1)
    pages, count = spa.new_page_pool(3, "cpu")
    assert pages.tolist() == [2, 1, 0] and count.tolist() == [3, 0] and pages.dtype == count.dtype == torch.int32
