"""The cache, attention and norm calls make their tensors' device the current one before they launch and give it back (CPU
only: the device switch is recorded, and a host without a GPU ends every call before its launch)."""
import os
import shutil
import subprocess
import sys
import sysconfig

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))

# Each call in a process of its own kind: the recorder takes the place of torch's device switch for good.
PROGRAM = """
import sys
sys.path[:0] = [{build!r}, {root!r}]
import torch
import device_recorder as R
import activation_sparsification_amd as spa
R.install()
bf, i32, u8 = torch.bfloat16, torch.int32, torch.uint8
def f(*shape, dtype=bf): return R.fake(shape, dtype, 1)
q, kv, cu = f(2, 4, 64), f(2, 2, 64), f(2, dtype=i32)
cache = spa.KvCache(f(2, 2, 16, 64), f(2, 2, 16, 64))
need = spa.lib().spa_attention_decode_workspace_bytes(2, 4, 2, 64)
ws = f(need, dtype=u8) if need <= 65536 else f(65536, dtype=u8)
calls = dict(
    kv_write=lambda: spa.kv_write(kv, kv, f(2, dtype=i32), cache),
    kv_read=lambda: spa.kv_read(cache, f(1, 2, dtype=i32), cu, 2, k_out=kv, v_out=kv),
    attention_decode=lambda: spa.attention_decode(q, cache, f(2, 2, dtype=i32), f(2, dtype=i32), out=q, ws=ws),
    attention_prefill=lambda: spa.attention_prefill(q, kv, kv, cu, out=q),
    gated_residual_norm=lambda: spa.gated_residual_norm(f(2, 64), f(2, 64), h_out=f(2, 64), y_out=f(2, 64)))
R.switches()
for name, call in calls.items():
    try:
        call()
        print(name, 'launched')
    except RuntimeError:
        print(name, *R.switches())
"""


def test_calls_switch_to_their_tensors_device(tmp_path):
    import torch
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
    r = subprocess.run([sys.executable, "-c", PROGRAM.format(build=str(tmp_path), root=os.path.dirname(HERE))],
                       capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr
    got = {w[0]: w[1:] for w in (line.split() for line in r.stdout.splitlines()) if w}
    assert sorted(got) == ["attention_decode", "attention_prefill", "gated_residual_norm", "kv_read", "kv_write"], r.stdout
    for name, seen in got.items():
        assert seen == ["1", "0"], f"{name}: devices made current: {seen}"
