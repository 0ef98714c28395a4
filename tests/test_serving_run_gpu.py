"""A server's calls one after the other: pages and offsets from request lengths, the norm and rotation that fill the cache, and
attention over it; prompts, later pieces of them and captured steps of single tokens, with requests that end and begin.

What the calls pass on is held against bookkeeping in plain Python (tests/plan_ref.py) and a second cache whose sequences lie
one behind the other, written apart; attention against 64 bits over what that cache stands for (tests/attention_bounds.py).
"""
import pytest
import torch

import attention_bounds as A
import mxfp4_ref as M
import plan_ref as P
from test_cache4_gpu import query_error

pytestmark = pytest.mark.gpu

spa = pytest.importorskip("activation_sparsification_amd")

I32 = torch.int32
N, WIDTH, PAGE, HQ, HKV = 4, 12, 16, 8, 2
CAP = WIDTH * PAGE


class Server:
    def __init__(self, dev, fmt, d, dtype, n_pages):
        self.dev, self.fmt, self.d, self.dtype = dev, fmt, d, dtype
        self.g = torch.Generator(device=dev).manual_seed(d)
        self.cache = spa.new_kv_cache(n_pages, PAGE, HKV, d, dtype, fmt, dev)
        self.mirror = spa.new_kv_cache(N * WIDTH, PAGE, HKV, d, dtype, fmt, dev)
        self.pool, self.count = spa.new_page_pool(n_pages, dev)
        self.table = torch.full((N, WIDTH), -1, dtype=I32, device=dev)
        self.lens = torch.zeros(N, dtype=I32, device=dev)
        self.books = dict(lens=[0] * N, table=self.table.tolist(), stack=self.pool.tolist(), count=[n_pages, 0])
        self.freq = 10000.0 ** (-torch.arange(d // 2, device=dev) / (d // 2))
        self.w = [(1 + 0.2 * torch.randn(d, generator=self.g, device=dev)).to(dtype) for _ in range(2)]

    def rows(self, t):
        return torch.randn((t, HQ + 2 * HKV, self.d), generator=self.g, device=self.dev).to(self.dtype)

    def split(self, x):
        return x[:, :HQ], x[:, HQ:HQ + HKV], x[:, HQ + HKV:]

    def plan(self, new, t, done):
        return spa.kv_plan(self.lens, new, self.table, PAGE, self.pool, self.count, t, done=done, lens_out=self.lens, count_out=self.count)

    def embed(self, x, pos, slots, **k_out):
        q, k, v = self.split(x)
        return spa.qk_norm_rope(q, k, pos, self.freq, q_weight=self.w[0], k_weight=self.w[1], v=v, slots=slots, cache=self.cache, **k_out)

    def follow(self, x, new, t, done, got):
        """Holds a plan's results to the books and writes the rows into the second cache; the queries as computed apart."""
        b = self.books
        want = P.plan(b["lens"], new, b["table"], PAGE, b["stack"], b["count"][0], t, done)
        for name, y in zip(("slots", "positions", "cu_q", "cu_k", "lens", "count"), got):
            assert y.tolist() == want[name], name
        assert self.table.tolist() == want["table"] and self.pool.tolist() == want["stack"]
        self.books = want
        seqs = [s for s in range(N) for _ in range(new[s])]
        place = [s * CAP + p for s, p in zip(seqs, want["positions"])] + [-1] * (t - len(seqs))
        q, k, v = self.split(x)
        qo, ko = spa.qk_norm_rope(q, k, got[1], self.freq, q_weight=self.w[0], k_weight=self.w[1])
        spa.kv_write(ko, v, torch.tensor(place, dtype=I32, device=self.dev), self.mirror)
        return qo

    def held(self):
        """What the second cache stands for: keys and values [N, CAP, HKV, d] in float64."""
        out = []
        for c, s in ((self.mirror.k, self.mirror.k_scale), (self.mirror.v, self.mirror.v_scale)):
            x = M.values(c, s) if self.fmt == "mxfp4" else c.double() if s is None else c.float().double() * s.double()[..., None]
            out.append(x.view(N, WIDTH, HKV, PAGE, self.d).transpose(2, 3).reshape(N, CAP, HKV, self.d))
        return out

    def check_decode(self, out, q):
        k, v = self.held()
        for s, n in enumerate(self.books["lens"]):
            r = A.reference(q[s:s + 1], k[s, :n], v[s, :n], self.d ** -0.5, torch.ones((1, n), dtype=torch.bool, device=self.dev))
            if self.fmt == "mxfp4":
                r["ds"] = r["ds"] + query_error(q[s:s + 1], k[s, :n], self.d ** -0.5)
            A.check(out[s:s + 1], None, r, self.dtype, codes=self.fmt != "native")

    def prompt(self, new, t, done=None):
        x = self.rows(t)
        plan = self.plan(torch.tensor(new, dtype=I32, device=self.dev), t, None if done is None else torch.tensor(done, dtype=I32, device=self.dev))
        slots, pos, cu_q, cu_k = plan[:4]
        q, _ = self.embed(x, pos, slots)
        assert torch.equal(q, self.follow(x, new, t, done, plan))
        total = sum(self.books["lens"])
        k, v = spa.kv_read(self.cache, self.table, cu_k, total, dtype=self.dtype)
        for got, want in zip((k, v), self.held()):
            want = torch.cat([want[s, :n] for s, n in enumerate(self.books["lens"])])
            assert torch.equal(got, want.to(self.dtype))
        # queries behind the last sequence belong to none
        out = spa.attention_prefill(q[:sum(new)], k, v, cu_q, cu_k)[0]
        at, to = 0, 0
        for n, m in zip(new, self.books["lens"]):
            i, j = torch.arange(n, device=self.dev)[:, None], torch.arange(m, device=self.dev)[None]
            A.check(out[at:at + n], None, A.reference(q[at:at + n], k[to:to + m], v[to:to + m], self.d ** -0.5, j <= i + m - n), self.dtype)
            at, to = at + n, to + m


@pytest.mark.parametrize("fmt,d,dtype", [("mxfp4", 128, torch.bfloat16), ("mxfp4", 64, torch.float16), ("mxfp4", 96, torch.bfloat16),
                                         ("native", 128, torch.bfloat16), ("fp8", 64, torch.bfloat16), ("int8", 128, torch.float16)])
def test_prompts_and_captured_steps(fmt, d, dtype):
    dev = torch.device("cuda:0")
    s = Server(dev, fmt, d, dtype, n_pages=30)
    s.prompt([37, 0, 5, 64], t=120)
    s.prompt([3, 20, 0, 1], t=24)
    x, ones, done = s.rows(N), torch.ones(N, dtype=I32, device=dev), torch.zeros(N, dtype=I32, device=dev)
    state = (s.lens, s.count, s.table, s.pool, *(y for y in (s.cache.k, s.cache.v, s.cache.k_scale, s.cache.v_scale) if y is not None))

    def step():
        plan = s.plan(ones, N, done)
        q, _ = s.embed(x, plan[1], plan[0])
        return plan, q, spa.attention_decode(q, s.cache, s.table, plan[4])[0]

    kept = [y.clone() for y in state]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    for y, old in zip(state, kept):
        y.copy_(old)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        plan, q, out = step()
    for i in range(20):
        x.copy_(s.rows(N))
        ended = [int(i == 3), int(i == 9), 0, int(i in (3, 12))]
        done.copy_(torch.tensor(ended, dtype=I32))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(q, s.follow(x, [1] * N, N, ended, plan))
        s.check_decode(out, q)
        if i == 10:
            s.prompt([16, 0, 7, 0], t=23, done=[0, 0, 1, 0])


def test_two_servers_on_two_streams():
    # the same calls on two streams at once, each with its own cache and pool, are what they are alone
    dev = torch.device("cuda:0")

    def step(server, x):
        plan = server.plan(server.ones, N, None)
        q, _ = server.embed(x, plan[1], plan[0])
        server.outs.append(spa.attention_decode(q, server.cache, server.table, plan[4])[0])

    def build():
        s = Server(dev, "mxfp4", 128, torch.bfloat16, 30)
        s.ones, s.outs = torch.ones(N, dtype=I32, device=dev), []
        return s, [s.rows(N) for _ in range(40)]

    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    pairs = [build(), build()]
    alone, rows = build()
    torch.cuda.synchronize()
    for i in range(40):
        for (s, xs), st in zip(pairs, streams):
            with torch.cuda.stream(st):
                step(s, xs[i])
    torch.cuda.synchronize()
    for x in rows:
        step(alone, x)
    torch.cuda.synchronize()
    for s, _ in pairs:
        assert all(torch.equal(a, b) for a, b in zip(s.outs, alone.outs))
        assert torch.equal(s.cache.k, alone.cache.k) and s.lens.tolist() == [40] * N
