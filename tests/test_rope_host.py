"""The norm and rotation of queries and keys on the host (CPU only): refusals through the C ABI before any launch."""
import ctypes
import math

import pytest

OK, INVALID, UNSUPPORTED = 0, 1, 2


@pytest.fixture(scope="module")
def B():
    import activation_sparsification_amd._binding as b
    b.lib()
    return b


def test_refusals(B):
    L = B.lib()

    def heads(data=4096, row=1024, head=64):
        return B._Heads(data, row, head)

    def cache(dtype=2, fmt=0, h=2, d=64, k=4096, ks=None):
        return B._KvCache(dtype, fmt, 4, 16, h, d, k, 8192, ks, ks)

    def call(q=heads(), k=heads(), v=None, dtype=2, t=4, hq=8, hkv=2, d=64, pos=4096, rope=B._Rope(4096, 64, 0), qn=None, kn=None,
             eps=1e-5, qo=heads(65536), ko=heads(131072), slots=None, c=None):
        return L.qk_norm_rope(q, k, v, dtype, t, hq, hkv, d, pos, rope, qn, kn, eps, qo, ko, slots, c, None)

    cached = dict(v=heads(), slots=256, c=cache())
    assert call(t=0) == OK and call(t=0, q=None, k=None, qo=None, ko=None, pos=None) == OK
    bad = B._Norm(4, None, None)
    for kw in (dict(dtype=7), dict(t=-1), dict(hq=0), dict(hkv=0), dict(hq=1 << 13), dict(d=0), dict(eps=-1.0), dict(eps=math.nan),
               dict(eps=math.inf), dict(q=None), dict(k=heads(None)), dict(qo=None), dict(ko=None), dict(qo=heads(None)),
               dict(q=heads(row=-8)), dict(k=heads(head=(1 << 23) + 8)), dict(pos=None), dict(rope=B._Rope(None, 64, 0)),
               dict(rope=B._Rope(4096, 66, 0)), dict(rope=B._Rope(4096, -2, 0)), dict(rope=B._Rope(4096, 7, 0)), dict(qn=bad), dict(kn=bad),
               dict(qn=B._Norm(1, 4100, None)), dict(kn=B._Norm(1, None, 4104)),
               dict(qo=heads(row=0)), dict(qo=heads(head=0)), dict(qo=heads(row=256)), dict(ko=heads(row=64)), dict(ko=heads(head=32)),
               dict(v=heads()), dict(slots=256), dict(cached, v=None), dict(cached, slots=None), dict(cached, c=cache(dtype=1)),
               dict(cached, c=cache(h=4)), dict(cached, c=cache(d=128)), dict(cached, c=cache(fmt=1)), dict(cached, c=cache(fmt=5)),
               dict(cached, c=cache(k=None)), dict(cached, ko=heads(row=0))):
        assert call(**kw) == INVALID, kw
    for kw in (dict(dtype=0), dict(d=60, rope=None), dict(rope=B._Rope(4096, 12, 0)), dict(rope=B._Rope(4096, 4, 1)), dict(q=heads(4104)),
               dict(k=heads(row=1028)), dict(qo=heads(65544)), dict(ko=heads(131072, 1024, 68)), dict(t=1 << 24),
               dict(cached, v=heads(4104))):
        assert call(**kw) == UNSUPPORTED, kw
    # one row, or one head: the stride of that axis is not used
    assert call(t=0, qo=heads(row=0)) == OK
    assert call(q=heads(4104), t=1, qo=heads(65536, 0, 64), ko=heads(131072, 0, 64)) == UNSUPPORTED


def test_rope_descriptor(B):
    assert ctypes.sizeof(B._Rope) == 16
