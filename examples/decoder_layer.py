"""A small decoder with pruned linear layers, run on a batch of prompts and then token by token.

Each layer is the library's calls in the order a server makes them: norm, pruned QKV projection, cache write,
attention, pruned output projection, gated residual norm, pruned squared-ReLU FFN, gated residual norm.  Prompts of
different lengths run packed, a second piece of each prompt attends to its cached beginning, and single tokens run
over the paged cache.  The result of the last token is compared with running every sequence whole.

With --rotate queries and keys are normed and turned by their positions on the way to the attention and into the cache;
with --pool pages come from a stack of free ones, and slots, positions and offsets are made on the GPU.

    python examples/decoder_layer.py --format mxfp4 --rotate --pool
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import activation_sparsification_amd as spa  # noqa: E402


class Layer:
    """Weights of one decoder layer and its part of the cache."""

    def __init__(self, g, hidden, ffn, heads, kv_heads, head_dim, n_pages, page, fmt, dtype, dev, rotate=False):
        def weight(n_out, k):
            w = torch.randn((n_out, k), generator=g, device=dev) * k ** -0.5
            return spa.prepare_weight(w.to(dtype), alpha=0.5)

        def vector(mean, std, size=hidden):
            return (mean + std * torch.randn(size, generator=g, device=dev)).to(dtype)

        self.heads, self.kv_heads, self.head_dim = heads, kv_heads, head_dim
        self.qkv = weight((heads + 2 * kv_heads) * head_dim, hidden)
        self.out, self.up, self.down = weight(hidden, heads * head_dim), weight(ffn, hidden), weight(hidden, ffn)
        self.post = [vector(1.0, 0.1) for _ in range(2)]
        self.pre = [vector(1.0, 0.1) for _ in range(2)]
        self.gate = [vector(0.5, 0.1) for _ in range(2)]
        self.qk = [vector(1.0, 0.1, head_dim) for _ in range(2)] if rotate else None
        self.cache = spa.new_kv_cache(n_pages, page, kv_heads, head_dim, dtype, fmt, dev)


class Decoder:
    """Layers, the page tables of a batch of sequences and their lengths."""

    def __init__(self, n_seqs, longest, layers=2, hidden=512, ffn=1024, heads=8, kv_heads=2, head_dim=64, page=16,
                 fmt="native", dtype=torch.bfloat16, dev="cuda", seed=0, rotate=False, pool=False):
        g = torch.Generator(device=dev)
        g.manual_seed(seed)
        width = -(-longest // page)
        self.layers = [Layer(g, hidden, ffn, heads, kv_heads, head_dim, n_seqs * width, page, fmt, dtype, dev, rotate)
                       for _ in range(layers)]
        # pages in no order, as an allocator hands them out
        self.table = torch.randperm(n_seqs * width, generator=g, device=dev).to(torch.int32).view(n_seqs, width)
        self.lens = torch.zeros(n_seqs, dtype=torch.int32, device=dev)
        self.page, self.hidden, self.dev = page, hidden, dev
        self.freq = 10000.0 ** (-torch.arange(0, head_dim, 2, device=dev) / head_dim) if rotate else None
        self.pool = spa.new_page_pool(n_seqs * width, dev) if pool else None
        if pool:
            self.table.fill_(-1)
        self.cfg = spa.PruneConfig(8, 16, score="weight", shift="token_mean")
        self.cfg_act = spa.PruneConfig(8, 16, score="weight", shift="token_mean", act="relu2")

    def _slots(self, seq, pos):
        return (self.table[seq, pos // self.page].long() * self.page + pos % self.page).to(torch.int32)

    def _plan(self, new, t):
        """Pages for ``new[s]`` more tokens of each sequence: slots, positions, cu_q, cu_k; the lengths move on."""
        pages, count = self.pool
        return spa.kv_plan(self.lens, new, self.table, self.page, pages, count, t, lens_out=self.lens, count_out=count)[:4]

    def _run(self, x, pos, slots, attend, linear):
        """Rows x [t, hidden] through every layer; ``attend(layer, q, k, v)`` is the attention of this kind of call."""
        h, y = spa.gated_residual_norm(x, None, pre="rms", pre_weight=self.layers[0].pre[0])
        h = h.float()                                           # the residual stream is kept in float32
        for i, layer in enumerate(self.layers):
            qkv, _, _ = linear(y, layer.qkv, self.cfg)
            qkv = qkv.view(x.shape[0], -1, layer.head_dim)
            q, k, v = qkv.split([layer.heads, layer.kv_heads, layer.kv_heads], dim=1)
            if self.freq is None:
                spa.kv_write(k, v, slots, layer.cache)
            else:
                q, k = spa.qk_norm_rope(q, k, pos, self.freq, q_weight=layer.qk[0], k_weight=layer.qk[1], q_out=q, k_out=k, v=v,
                                        slots=slots, cache=layer.cache)
            a = attend(layer, q, k, v)
            o, _, _ = linear(a.view(x.shape[0], -1), layer.out, self.cfg)
            h, y = spa.gated_residual_norm(o, h, post="rms", post_weight=layer.post[0], gate=layer.gate[0], scale=0.5,
                                           pre="rms", pre_weight=layer.pre[1], h_out=h, y_out=o)
            u, _, _ = linear(y, layer.up, self.cfg)
            f, _, _ = linear(u, layer.down, self.cfg_act)       # the squared ReLU is applied inside the call
            nxt = self.layers[i + 1].pre[0] if i + 1 < len(self.layers) else None
            h, y = spa.gated_residual_norm(f, h, post="rms", post_weight=layer.post[1], gate=layer.gate[1], scale=0.5,
                                           pre="rms", pre_weight=nxt, h_out=h, y_out=f)
        return y

    def prompt(self, x, new):
        """The next ``new[s]`` tokens of each sequence, packed in x; what is cached already is attended to."""
        new = torch.tensor(new, dtype=torch.int32, device=self.dev)
        fresh = not bool(self.lens.any())
        if self.pool:
            slots, pos, cu_q, cu_k = self._plan(new, x.shape[0])
        else:
            slots, pos, cu_q, cu_k = self._offsets(new, x.shape[0])
        total = int(cu_k[-1])

        def attend(layer, q, k, v):
            if not fresh:                                       # the cached beginning and the new piece, as dense rows
                k, v = spa.kv_read(layer.cache, self.table, cu_k, total, dtype=q.dtype)
            return spa.attention_prefill(q, k, v, cu_q, cu_q if fresh else cu_k)[0]

        return self._run(x, pos, slots, attend, spa.sparse_linear_prefill)

    def _offsets(self, new, t):
        """What ``_plan`` gives, in torch operations over a table that is filled from the start."""
        cu_q = torch.nn.functional.pad(new.cumsum(0), (1, 0)).to(torch.int32)
        have = self.lens + new
        cu_k = torch.nn.functional.pad(have.cumsum(0), (1, 0)).to(torch.int32)
        seq = torch.repeat_interleave(torch.arange(len(new), device=self.dev), new.long())
        pos = torch.arange(t, device=self.dev) - cu_q[:-1].long()[seq] + self.lens.long()[seq]
        self.lens = have
        return self._slots(seq, pos), pos.to(torch.int32), cu_q, cu_k

    def step(self, x):
        """One new token of each sequence, x [n_seqs, hidden] (up to 32 sequences)."""
        new = torch.ones(x.shape[0], dtype=torch.int32, device=self.dev)
        slots, pos = (self._plan if self.pool else self._offsets)(new, x.shape[0])[:2]

        def attend(layer, q, k, v):
            return spa.attention_decode(q, layer.cache, self.table, self.lens)[0]

        return self._run(x, pos, slots, attend, spa.sparse_linear_decode)


def compare(fmt="native", lens=(70, 33, 129), pieces=20, steps=3, seed=0, rotate=False, pool=False):
    """The last token's outputs after prompts, second pieces and single tokens, and after whole prompts: their relative
    difference in the 2-norm, one number per sequence."""
    longest = max(lens) + pieces + steps
    args = dict(n_seqs=len(lens), longest=longest, fmt=fmt, seed=seed, rotate=rotate, pool=pool)
    a, b = Decoder(**args), Decoder(**args)
    g = torch.Generator(device="cuda")
    g.manual_seed(seed + 1)
    full = [torch.randn((n + pieces + steps, a.hidden), generator=g, device="cuda").to(torch.bfloat16) for n in lens]
    a.prompt(torch.cat([x[:n] for x, n in zip(full, lens)]), list(lens))
    a.prompt(torch.cat([x[n:n + pieces] for x, n in zip(full, lens)]), [pieces] * len(lens))
    for i in range(steps):
        last = a.step(torch.stack([x[n + pieces + i] for x, n in zip(full, lens)]))
    whole = b.prompt(torch.cat(full), [x.shape[0] for x in full])
    ends = torch.tensor([x.shape[0] for x in full], device="cuda").cumsum(0) - 1
    want = whole[ends].double()
    return ((last.double() - want).norm(dim=-1) / want.norm(dim=-1)).tolist()


def main():
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--format", choices=["native", "fp8", "int8", "mxfp4"], default="native", help="how the cache holds vectors")
    ap.add_argument("--steps", type=int, default=3, help="single tokens after the prompts")
    ap.add_argument("--rotate", action="store_true", help="norm and turn queries and keys")
    ap.add_argument("--pool", action="store_true", help="pages from a pool, planned on the GPU")
    args = ap.parse_args()
    got = compare(args.format, steps=args.steps, rotate=args.rotate, pool=args.pool)
    print(f"cache {args.format}: last token against whole prompts, relative difference "
          + ", ".join(f"{x:.2e}" for x in got))


if __name__ == "__main__":
    main()
