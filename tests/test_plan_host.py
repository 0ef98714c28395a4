"""Page planning on the host (CPU only): refusals through the C ABI before any launch, and the reference's own invariants."""
import ctypes
import random

import pytest

import plan_ref as P

OK, INVALID, UNSUPPORTED = 0, 1, 2


@pytest.fixture(scope="module")
def B():
    import activation_sparsification_amd._binding as b
    b.lib()
    return b


def test_refusals(B):
    L = B.lib()

    def pool(pages=4096, count=512, out=1024, n=8):
        return B._PagePool(pages, count, out, n)

    def call(lens=16, fresh=32, done=None, n=3, table=64, width=4, page=16, p=pool(), t=5, slots=128, pos=256, cq=384, ck=640, lo=768):
        return L.spa_kv_plan(lens, fresh, done, n, table, width, page, p, t, slots, pos, cq, ck, lo, None)

    for kw in (dict(n=-1), dict(n=(1 << 20) + 1), dict(width=-1), dict(page=0), dict(page=-3), dict(t=-1), dict(t=(1 << 30) + 1), dict(p=None),
               dict(p=pool(n=-1)), dict(p=pool(pages=None)), dict(p=pool(count=None)), dict(p=pool(out=None)), dict(lens=None), dict(fresh=None),
               dict(lo=None), dict(lo=32), dict(table=None), dict(slots=None), dict(pos=None), dict(pos=128), dict(cq=None), dict(ck=None),
               dict(ck=384)):
        assert call(**kw) == INVALID, kw
    for kw in (dict(width=1 << 26), dict(page=1 << 28), dict(p=pool(n=1 << 28))):
        assert call(**kw) == UNSUPPORTED, kw
    assert ctypes.sizeof(B._PagePool) == 32


def test_reference_keeps_every_page(B):
    rng = random.Random(1)
    stack, table, lens, count = list(range(40)), [[-1] * 8 for _ in range(6)], [0] * 6, 40
    for _ in range(200):
        new, done = [rng.randint(0, 5) for _ in lens], [int(x > 20) for x in lens]
        r = P.plan(lens, new, table, 4, stack, count, 30, done)
        used = [p for row, x in zip(r["table"], r["lens"]) for p in row[:-(-x // 4)] if p >= 0]
        assert sorted(used + r["stack"][:r["count"][0]]) == list(range(40))
        live = [x for x in r["slots"] if x >= 0]
        assert len(set(live)) == len(live)
        stack, table, lens, count = r["stack"], r["table"], r["lens"], r["count"][0]
