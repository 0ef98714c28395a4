"""Where the norm and rotation of queries and keys may write, on the host (CPU only): its overlap check against marked bytes, and
the calls on a packed projection that are refused before any launch, through the C ABI."""
import os
import shutil
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
INVALID = 1


def test_overlaps_under_sanitizers(tmp_path):
    cxx = shutil.which("g++")
    if cxx is None:
        pytest.skip("no host C++ compiler")
    exe = str(tmp_path / "rope_overlap_driver")
    cmd = [cxx, "-std=c++17", "-O1", "-g", "-fsanitize=address,undefined", "-fno-sanitize-recover=undefined", "-Wall",
           "-I", os.path.join(ROOT, "include"), "-I", os.path.join(ROOT, "activation_sparsification_amd", "csrc"),
           os.path.join(HERE, "native", "rope_overlap_driver.cpp"), "-o", exe]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0 and "sanitizer" in r.stderr.lower():
        pytest.skip("no sanitizer runtime for the host compiler")
    assert r.returncode == 0, r.stderr
    r = subprocess.run([exe], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stdout + r.stderr
    words = r.stdout.split()
    assert words[0] == "ok" and int(words[2]) > 10000 and int(words[1]) - int(words[2]) > 10000, r.stdout


# Offsets in heads from the start of a packed projection x [4, 12, 64] (8 query, 2 key, 2 value heads); y: another buffer.
@pytest.mark.parametrize("q_out,k_out,cached", [(("x", 1), ("x", 8), False), (("x", 1), ("y", 8), False), (("x", 1), None, True),
                                                (("y", 0), ("y", 7), False), (("y", 2), ("y", 1), True), (("x", 0), ("x", 9), False),
                                                (("x", 0), ("x", 9), True), (("x", 12), ("y", 8), False), (("x", 10), None, True),
                                                (("x", 5), ("y", 8), True)])
def test_packed_views_are_refused(q_out, k_out, cached):
    import activation_sparsification_amd._binding as b
    base = {"x": 1 << 20, "y": 1 << 21}

    def heads(at):
        return b._Heads(base[at[0]] + 2 * 64 * at[1], 12 * 64, 64)

    cache = b._KvCache(2, 0, 4, 16, 2, 64, 1 << 22, 1 << 23, None, None) if cached else None
    got = b.lib().qk_norm_rope(heads(("x", 0)), heads(("x", 8)), heads(("x", 10)) if cached else None, 2, 4, 8, 2, 64, 4096,
                               b._Rope(8192, 64, 0), None, None, 1e-5, heads(q_out), heads(k_out) if k_out else None,
                               16384 if cached else None, cache, None)
    assert got == INVALID
