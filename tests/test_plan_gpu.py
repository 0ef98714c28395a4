"""Page tables, slots and offsets from request lengths on the GPU, number for number against tests/plan_ref.py."""
import random

import pytest
import torch

import plan_ref as P

pytestmark = pytest.mark.gpu

spa = pytest.importorskip("activation_sparsification_amd")

I32 = torch.int32
NAMES = ("slots", "positions", "cu_q", "cu_k", "lens", "count")


@pytest.fixture(scope="module")
def dev():
    assert torch.cuda.is_available(), "GPU tests need a device"
    return torch.device("cuda:0")


def state(rng, lens, page, width, n_pages):
    """A table whose sequences own distinct pages, the free ones on a stack."""
    pages = list(range(n_pages))
    rng.shuffle(pages)
    table = []
    for x in lens:
        need = -(-min(max(x, 0), width * page) // page)
        table.append([pages.pop() for _ in range(need)] + [rng.choice([-1, 7, 2 ** 31 - 1]) for _ in range(width - need)])
    return table, pages + [-3] * (n_pages - len(pages)), len(pages)


def ints(x, dev, shape=None):
    t = torch.tensor(x, dtype=I32, device=dev)
    return t if shape is None else t.reshape(shape)


def run(dev, lens, new, table, page, stack, count, t, done=None, inplace=False):
    n, width = len(lens), len(table[0]) if table else 0
    want = P.plan(lens, new, table, page, stack, count, t, done)
    args = [ints(lens, dev), ints(new, dev), ints(table, dev, (n, width)), page, ints(stack, dev), ints([count, 99], dev), t]
    given = {}
    if inplace:
        given = dict(lens_out=args[0], count_out=args[5])
    got = dict(zip(NAMES, spa.kv_plan(*args, done=None if done is None else ints(done, dev), **given)))
    if inplace:
        assert got["lens"] is args[0] and got["count"] is args[5]
    else:
        assert args[0].tolist() == lens and args[5].tolist() == [count, 99]
    got.update(table=args[2], stack=args[4])
    for name, x in want.items():
        assert got[name].tolist() == x, name
    return want


@pytest.mark.parametrize("inplace", [False, True])
@pytest.mark.parametrize("n,longest,most_new,page,seed", [(1, 1, 1, 1, 0), (1, 100, 3000, 16, 1), (64, 4000, 1, 16, 2), (7, 50, 9, 7, 3), (200, 300, 40, 16, 4),
                                                          (3, 5000, 2500, 64, 5), (700, 30, 2, 1, 6), (40, 900, 300, 100, 7), (2, 0, 2048, 32, 8),
                                                          (2500, 60, 5, 16, 9)])
def test_steps(dev, inplace, n, longest, most_new, page, seed):
    rng = random.Random(seed)
    for pad, over in ((0, 0.0), (3, 0.2), (1000, 1.0)):
        lens = [rng.randint(0, longest) for _ in range(n)]
        new = [0 if rng.random() < 0.2 else rng.randint(1, most_new) for _ in range(n)]
        done = [int(rng.random() < over) for _ in range(n)] if over else None
        width = -(-(longest + most_new) // page)
        n_pages = sum(-(-x // page) for x in lens) + sum(-(-x // page) + 1 for x in new)
        run(dev, lens, new, *with_page(state(rng, lens, page, width, n_pages), page), sum(new) + pad, done, inplace)


def with_page(s, page):
    return s[0], page, s[1], s[2]


@pytest.mark.parametrize("inplace", [False, True])
def test_too_few_pages(dev, inplace):
    rng = random.Random(3)
    for n_free in (0, 1, 5, 40):
        lens, new = [rng.randint(0, 50) for _ in range(30)], [rng.randint(0, 20) for _ in range(30)]
        held = sum(-(-x // 8) for x in lens)
        table, stack, count = state(rng, lens, 8, 10, held + n_free)
        got = run(dev, lens, new, table, 8, stack, count, sum(new) + 4, None, inplace)
        assert count == n_free and (got["count"][1] > 0) == (n_free < 40)
        # the next step finds the columns without a page, and gives back what there is
        more = [1] * 30
        run(dev, got["lens"], more, got["table"], 8, got["stack"], got["count"][0], 30, [1, 0] * 15, inplace)


def test_rows_that_do_not_fit_are_cut_off(dev):
    rng = random.Random(4)
    lens, new = [5, 0, 33, 2], [10, 3000, 0, 50]
    for t in (0, 1, 9, 10, 11, 2047, 2048, 2049, 3010, 3059, 3060, 5000):
        table, stack, count = state(rng, lens, 16, 300, 300)
        run(dev, lens, new, table, 16, stack, count, t)
        run(dev, lens, new, table, 16, stack, count, t, [0, 1, 1, 0], True)


def test_numbers_out_of_range(dev):
    rng = random.Random(5)
    top = 2 ** 31 - 1
    table, stack, count = state(rng, [20, 20, 20, 20], 16, 4, 30)
    for lens, new in (([-5, top, 20, 64], [3, 4, -7, 9]), ([20, 63, 64, 65], [1, 2, 3, -top]), ([0, 20, 1, 2], [top, top, top, top])):
        for done in (None, [1, 0, 1, 0], [-1, 5, 0, top]):
            run(dev, lens, new, table, 16, stack, count, 150, done)
    run(dev, [20, 20, 20, 20], [9, 9, 20, 20], table, 16, stack, 31, 60)            # a count above the stack, and below
    run(dev, [20, 20, 20, 20], [9, 9, 20, 20], table, 16, stack, -4, 60)
    bad = list(stack)
    bad[count - 1], bad[count - 2], bad[count - 3] = 30, -7, top                    # entries that are no pages
    run(dev, [20, 20, 20, 20], [20, 20, 20, 20], table, 16, bad, count, 80)
    gaps = [list(r) for r in table]
    gaps[1][0], gaps[2][1] = -1, 30                                                 # columns without a page are not given back
    run(dev, [20, 20, 20, 20], [1, 1, 1, 1], gaps, 16, stack, count, 4, [1, 1, 1, 1])
    twice = [list(r) for r in table]
    twice[1] = list(table[0])                                                       # more given back than the stack holds
    run(dev, [64, 64, 20, 20], [0, 0, 0, 0], [[3, 3, 3, 3]] * 4, 16, stack, 28, 4, [1, 1, 1, 1])


def test_nothing_to_do(dev):
    run(dev, [], [], [], 16, [4, 2, 0], 3, 5)
    run(dev, [], [], [], 16, [], 0, 0)
    rng = random.Random(6)
    table, stack, count = state(rng, [7, 8], 4, 5, 12)
    run(dev, [7, 8], [0, 0], table, 4, stack, count, 0)
    run(dev, [7, 8], [2, 3], table, 4, [], 0, 5)                                    # no pages at all
    run(dev, [7, 8], [2, 3], [[], []], 4, stack, count, 5)                          # a table without columns
    got = spa.kv_plan(*[ints(x, dev) for x in ([], [])], torch.empty((0, 0), dtype=I32, device=dev), 16, ints([1], dev), ints([1, 0], dev), 3)
    assert [x.tolist() for x in got] == [[-1] * 3, [0] * 3, [0], [0], [], [1, 0]]


@pytest.mark.parametrize("n", [2047, 2048, 2049, 4100, 9000])
def test_many_sequences(dev, n):
    rng = random.Random(n)
    lens, new = [rng.randint(0, 9) for _ in range(n)], [rng.choice([0, 1, 1, 3]) for _ in range(n)]
    table, stack, count = state(rng, lens, 4, 3, 4 * n)
    done = [int(rng.random() < 0.3) for _ in range(n)]
    run(dev, lens, new, table, 4, stack, count, sum(new) + 1)
    run(dev, lens, new, table, 4, stack, count, sum(new), done, True)


def test_long_sequences(dev):
    # sums past 31 bits, offsets of the table's entries, thousands of columns of one sequence taken and given back
    n, width, page = 9, 30000, 16384
    lens = [width * page - 5 - i for i in range(n)]
    table = torch.arange(width, dtype=I32, device=dev).repeat(n, 1)
    pool, count = spa.new_page_pool(2 ** 17 - 1, dev)
    got = dict(zip(NAMES, spa.kv_plan(ints(lens, dev), ints([3] * n, dev), table, page, pool, count, 3 * n)))
    after = [x + 3 for x in lens]
    assert got["lens"].tolist() == after
    sums = [0]
    for x in after:
        sums.append(min(sums[-1] + x, P.TOP))
    assert got["cu_k"].tolist() == sums and sums[-1] == P.TOP
    assert got["positions"].tolist() == [x + i for x in lens for i in range(3)]
    assert got["slots"].tolist() == [(width - 1) * page + (x + i) % page for x in lens for i in range(3)]
    rng = random.Random(1)
    held, stack, free = state(rng, [70000, 3, 50000], 16, 5000, 9000)
    run(dev, [70000, 3, 50000], [9000, 0, 1], held, 16, stack, free, 9001, [0, 0, 1])
    run(dev, [70000, 3, 50000], [9000, 0, 1], held, 16, stack, free, 9001, [1, 1, 1], True)


def test_pool_runs_out_and_comes_back(dev):
    # a program's loop, everything in place: what is out of the pool stands in one row's used columns, and nowhere else
    rng = random.Random(8)
    n, width, page, n_pages = 12, 16, 4, 90
    pool, count = spa.new_page_pool(n_pages, dev)
    assert pool.tolist() == list(range(n_pages - 1, -1, -1)) and count.tolist() == [n_pages, 0]
    lens, table = torch.zeros(n, dtype=I32, device=dev), torch.full((n, width), -1, dtype=I32, device=dev)
    mirror = dict(lens=[0] * n, table=table.tolist(), stack=pool.tolist(), count=[n_pages, 0])
    for step in range(60):
        new = [rng.choice([0, 1, 1, 1, 9]) for _ in range(n)]
        done = [int(x + m > width * page or rng.random() < 0.05) for x, m in zip(mirror["lens"], new)]
        want = P.plan(mirror["lens"], new, mirror["table"], page, mirror["stack"], mirror["count"][0], 64, done)
        got = dict(zip(NAMES, spa.kv_plan(lens, ints(new, dev), table, page, pool, count, 64, done=ints(done, dev), lens_out=lens, count_out=count)))
        got.update(table=table, stack=pool)
        for name, x in want.items():
            assert got[name].tolist() == x, (step, name)
        mirror = want
        used = [p for r, x in zip(want["table"], want["lens"]) for p in r[:-(-x // page)] if p >= 0]
        assert sorted(used + want["stack"][:want["count"][0]]) == list(range(n_pages))


def test_captured_steps_advance(dev):
    # a captured step of single tokens replayed with its lengths, count and table in place, against the eager calls
    n, width, page = 33, 40, 4
    args = []
    for _ in range(2):
        pool, count = spa.new_page_pool(n * width, dev)
        args.append([torch.arange(n, dtype=I32, device=dev), torch.ones(n, dtype=I32, device=dev),
                     torch.full((n, width), -1, dtype=I32, device=dev), page, pool, count, 40])
    for a in args:                                      # the beginnings
        first = a[0].clone()
        a[0].zero_()
        spa.kv_plan(a[0], first, *a[2:6], int(first.sum()), lens_out=a[0], count_out=a[5])
    done = torch.zeros(n, dtype=I32, device=dev)

    def step(a):
        return spa.kv_plan(*a, done=done, lens_out=a[0], count_out=a[5])

    keep = [x.clone() for x in (args[0][0], args[0][2], args[0][4], args[0][5])]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(args[0])
    torch.cuda.current_stream().wait_stream(side)
    for x, old in zip((args[0][0], args[0][2], args[0][4], args[0][5]), keep):
        x.copy_(old)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step(args[0])
    for i in range(9):
        done.zero_()
        if i % 4 == 3:
            done[i::5] = 1
        graph.replay()
        want = step(args[1])
        torch.cuda.synchronize()
        for name, a, b in zip(NAMES, out, want):
            assert torch.equal(a, b), (i, name)
        assert torch.equal(args[0][2], args[1][2]) and torch.equal(args[0][4], args[1][4])


def test_given_outputs_and_slices(dev):
    # tensors that begin off 16 bytes
    rng = random.Random(2)
    lens, new = [3, 9, 0], [2, 1, 5]
    table, stack, count = state(rng, lens, 4, 5, 20)
    want = P.plan(lens, new, table, 4, stack, count, 9)
    off = lambda x: ints([0] + x, dev)[1:]
    whole = ints([[0] * 5] + table, dev)
    out = {name: ints([-9] * (len(want[name]) + 2), dev) for name in NAMES}
    given = {("count_out" if k == "count" else "lens_out" if k == "lens" else k): v[1:-1] for k, v in out.items()}
    got = spa.kv_plan(off(lens), off(new), whole[1:], 4, off(stack), off([count, 0]), 9, **given)
    for name, x in zip(NAMES, got):
        assert x.tolist() == want[name] and out[name][0] == -9 and out[name][-1] == -9, name
    assert whole[1:].tolist() == want["table"] and whole[0].tolist() == [0] * 5


def test_refusals(dev):
    i = lambda *s: torch.zeros(s, dtype=I32, device=dev)
    good = [i(3), i(3), i(3, 4), 16, i(8), i(2), 5]
    spa.kv_plan(*good)
    for at, bad, match in ((0, i(3).long(), "lens"), (0, i(3, 1), "lens"), (0, i(3).cpu(), "lens"), (1, i(2), "new"), (2, i(2, 4), "page_table"),
                           (2, i(12), "page_table"), (4, i(2, 4), "free_pages"), (5, i(1), "free_count"), (6, -1, "t: "), (2, i(3, 8)[:, :4], "page_table"),
                           (4, i(16)[::2], "free_pages")):
        args = list(good)
        args[at] = bad
        with pytest.raises(ValueError, match=match):
            spa.kv_plan(*args)
    for kw, match in ((dict(done=i(2)), "done"), (dict(done=torch.zeros(3, dtype=torch.bool, device=dev)), "done"), (dict(slots=i(4)), "slots"),
                      (dict(cu_q=i(3)), "cu_q"), (dict(lens_out=i(3).float()), "lens_out"), (dict(count_out=i(1)), "count_out")):
        with pytest.raises(ValueError, match=match):
            spa.kv_plan(*good, **kw)
    same = i(5)
    for kw in (dict(slots=same, positions=same),):
        with pytest.raises(spa.SpaError):
            spa.kv_plan(*good, **kw)
    for page in (0, -1, 2 ** 28):
        with pytest.raises(spa.SpaError):
            spa.kv_plan(*good[:3], page, *good[4:])


def test_writes_are_known_to_autograd(dev):
    table, pool = torch.full((2, 4), -1, dtype=I32, device=dev), spa.new_page_pool(8, dev)
    before = table._version, pool[0]._version, pool[1]._version
    lens = torch.zeros(2, dtype=I32, device=dev)
    spa.kv_plan(lens, lens + 3, table, 4, *pool, 6, lens_out=lens, count_out=pool[1])
    assert all(a > b for a, b in zip((table._version, pool[0]._version, pool[1]._version), before)) and lens._version > 0


def test_some_outputs_given(dev):
    # new outputs beside given ones, also where all that is new has no elements
    pool, count = spa.new_page_pool(4, dev)
    lens, new, table = ints([2], dev), ints([0], dev), ints([[1, -1]], dev)
    given = dict(cu_q=ints([9, 9], dev), cu_k=ints([9, 9], dev), lens_out=ints([9], dev), count_out=ints([9, 9], dev))
    got = dict(zip(NAMES, spa.kv_plan(lens, new, table, 4, pool, count, 0, **given)))
    assert got["slots"].shape == got["positions"].shape == (0,) and got["cu_k"].tolist() == [0, 2] and got["lens"].tolist() == [2]
    with torch.inference_mode():
        got = dict(zip(NAMES, spa.kv_plan(lens, new + 1, table, 4, pool, count, 2, cu_q=given["cu_q"])))
        got["slots"] += 1
    assert got["slots"].tolist() == [7, 0] and got["positions"].tolist() == [2, 0] and given["cu_q"].tolist() == [0, 1]
    got = dict(zip(NAMES, spa.kv_plan(lens, new, table, 4, pool, count, 3)))
    version = got["positions"]._version
    got["slots"].add_(1)
    assert got["positions"]._version == version and got["positions"].tolist() == [0, 0, 0] and got["slots"].tolist() == [0, 0, 0]


@pytest.mark.parametrize("inplace", [False, True])
@pytest.mark.parametrize("n,longest,most_new,t,page", [(1, 70, 5, 3, 16), (64, 300, 1, 64, 16), (65, 300, 1, 70, 16), (90, 200, 8, 512, 4), (90, 200, 12, 513, 4),
                                                       (211, 800, 60, 5000, 32), (513, 100, 3, 1500, 16), (600, 90, 7, 2049, 8), (2500, 40, 4, 9000, 16)])
def test_requests_that_end_and_begin(dev, inplace, n, longest, most_new, t, page):
    # over or not, with tokens in the same call or not; enough pages and too few; rows to spare and too few of them
    rng = random.Random(n + t)
    for few in (False, True):
        lens, new = [rng.randint(0, longest) for _ in range(n)], [rng.choice([0, 1, rng.randint(0, most_new)]) for _ in range(n)]
        done = [int(rng.random() < 0.3) for _ in range(n)]
        width = -(-(longest + most_new) // page)
        held = sum(-(-x // page) for x in lens)
        table, stack, count = state(rng, lens, page, width, held + (n // 8 if few else n * 3))
        run(dev, lens, new, table, page, stack, count, t // 2 if few else t, done, inplace)


def test_replaced_in_part(dev):
    # only the lengths, or only the count, in place, in calls of several workgroups
    rng = random.Random(5)
    for name, done in (("lens_out", None), ("count_out", None), ("lens_out", [0, 1, 0]), ("count_out", [1, 0, 0])):
        lens, new, page = [700, 20, 333], [900, 40, 800], 16
        table, stack, count = state(rng, lens, page, 120, 200)
        want = P.plan(lens, new, table, page, stack, count, 1800, done)
        args = [ints(lens, dev), ints(new, dev), ints(table, dev), page, ints(stack, dev), ints([count, 0], dev), 1800]
        given = {name: args[0] if name == "lens_out" else args[5]}
        got = dict(zip(NAMES, spa.kv_plan(*args, done=None if done is None else ints(done, dev), **given)))
        for key, x in want.items():
            assert {**got, "table": args[2], "stack": args[4]}[key].tolist() == x, (name, key)


def test_lengths_of_ended_requests(dev):
    # columns that fill a wave's loads, or all that it has in flight, and one more or fewer
    rng = random.Random(11)
    lens = [1, 63, 64, 65, 128, 129, 511, 512, 513, 575, 576, 577, 1024, 1088, 0, 2] * 2
    for gone in (range(32), range(0, 32, 3), [8], [13, 30]):
        table, stack, count = state(rng, lens, 1, 1100, sum(lens) + 40)
        run(dev, lens, [1] * 32, table, 1, stack, count, 32, [int(i in gone) for i in range(32)])
