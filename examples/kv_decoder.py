"""A small decoder whose attention keeps its keys and values in 4 bits (or 8) and whose
feed-forward layers are sparse MoE layers, run as a server would: prompts of different
lengths first, in one ragged batch, then single tokens, over the whole context or over the
pages that the cache's bounds choose; in 8 bits, over a cache that is kept at some tokens
per sequence by evicting those that attention has weighed least.

    python examples/kv_decoder.py [--steps 16] [--prompts 300,41,128] [--budget 0]
    python examples/kv_decoder.py --bits 8 [--keep 0]

Weights are random (seeded).  Needs a GPU and the built library."""
from __future__ import annotations

import argparse
import math
import os
import sys
import time

import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

from moe_expert_layer_sorted_gb300 import KVCache, KVCache8, harness  # noqa: E402
from synth import workloads as W  # noqa: E402


def norm(x):
    """Root-mean-square norm of the fp32 residual stream, in bf16."""
    return (x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6)).to(torch.bfloat16)


class Decoder:
    """`layers` times: attention over the cache, then the MoE layer; fp32 residual.  keep > 0 (8 bits): sequences of
    more than that many tokens go back to it after a step."""

    def __init__(self, layers=2, q_heads=8, kv_heads=2, head_dim=64, max_tokens=1024, sequences=4, context=2048, page_size=16,
                 seed=0, bits=4, keep=0):
        self.wl = W.WORKLOADS["tiny"]
        self.plan, _ = harness.build_plan(self.wl, max_tokens=max_tokens)
        hidden, g = self.wl.hidden, torch.Generator(device="cuda").manual_seed(seed)
        self.q_heads, self.kv_heads, self.head_dim, self.page_size = q_heads, kv_heads, head_dim, page_size

        def weight(rows, cols):
            return (torch.randn(rows, cols, generator=g, device="cuda") / math.sqrt(rows)).to(torch.bfloat16)

        wide = (q_heads + 2 * kv_heads) * head_dim
        self.qkv = [weight(hidden, wide) for _ in range(layers)]
        self.out = [weight(q_heads * head_dim, hidden) for _ in range(layers)]
        per_seq = -(-context // page_size)
        shape = dict(kv_heads=kv_heads, head_dim=head_dim, page_size=page_size, layers=layers)
        self.bits, self.keep = bits, keep
        if bits == 8:
            self.cache = KVCache8.allocate(sequences * per_seq, mass=keep > 0, **shape)
        else:
            self.cache = KVCache.allocate(sequences * per_seq, group_size=32, **shape)
        # pages are handed out in order here; a server would take them from a free list as sequences grow
        self.table = torch.arange(sequences * per_seq, dtype=torch.int32, device="cuda").view(sequences, per_seq)

    def close(self):
        self.cache.close()
        self.plan.close()

    def forward(self, x, lens, starts=None, max_new=None, budget=0):
        """x [rows, hidden] fp32: the new tokens' inputs, sequence after sequence; lens int32
        [sequences]: their lengths with the new tokens; starts, max_new: as for KVCache (None:
        one token each).  budget > 0: single tokens attend to that many pages.  Returns the
        new residual stream [rows, hidden]."""
        n, s = x.shape[0], lens.shape[0]
        batch = dict(table=self.table[:s], lens=lens)
        lead = (s, n // s) if starts is None else (n,)
        if starts is not None:
            batch.update(starts=starts, max_new=max_new)
        for layer, (wqkv, wout) in enumerate(zip(self.qkv, self.out)):
            heads = (norm(x) @ wqkv).view(*lead, -1, self.head_dim)
            q, k, v = heads.split((self.q_heads, self.kv_heads, self.kv_heads), dim=-2)  # views, read in place
            self.cache.append(k, v, layer=layer, **batch)
            o = torch.empty(*lead, self.q_heads, self.head_dim, dtype=torch.bfloat16, device="cuda")
            pages = None
            if budget:
                pages = torch.empty(n, self.kv_heads, budget, dtype=torch.int32, device="cuda")
                self.cache.select(q, pages, layer=layer, **batch)
            if self.bits == 8:
                weighed = dict(lse=torch.empty(n, self.q_heads, device="cuda"), weigh=True) if self.keep else {}
                self.cache.attention(q, o, layer=layer, **weighed, **batch)
            else:
                self.cache.attention(q, o, pages=pages, layer=layer, **batch)
            x = x + (o.view(n, -1) @ wout).float()
            h = norm(x)
            y, mixed = torch.empty_like(h), torch.empty_like(h)
            # the MoE layer with the residual added in its combine; the example keeps the stream in fp32
            self.plan.forward_residual(0, h, y, x, mixed)
            x = x + y.float()
        return x


    def evict(self, lens):
        """The lengths after every sequence of more than `keep` tokens has gone back to that many: the
        first few (which attention leans on), a quarter of the latest, and what weighed most."""
        if self.keep:
            kept = torch.empty(lens.shape[0], self.kv_heads, self.keep, dtype=torch.int32, device="cuda")
            for layer in range(len(self.qkv)):
                self.cache.evict(kept, table=self.table[:lens.shape[0]], lens=lens, keep_first=min(4, self.keep // 4),
                                 keep_last=max(self.keep // 4, 1), layer=layer)
            lens = lens.clamp_max(self.keep)
        return lens


def inputs(rows, hidden, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(rows, hidden, generator=g, device="cuda")


def run(prompts, steps, budget=0, decoder=None, seed=1):
    """Prompts, then `steps` single tokens of every sequence; returns the streams of the last
    prompt tokens and of every step."""
    d = decoder or Decoder()
    lens = torch.tensor(prompts, dtype=torch.int32, device="cuda")
    starts = torch.zeros(len(prompts) + 1, dtype=torch.int32, device="cuda")
    starts[1:] = torch.cumsum(lens, 0)
    x = d.forward(inputs(sum(prompts), d.wl.hidden, seed), lens, starts, max(prompts))
    outs = [x[starts[1:].long() - 1]]
    for i in range(steps):
        lens = d.evict(lens) + 1
        outs.append(d.forward(inputs(len(prompts), d.wl.hidden, seed + 1 + i), lens, budget=budget))
    return outs


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--steps", type=int, default=16)
    ap.add_argument("--prompts", default="300,41,128")
    ap.add_argument("--budget", type=int, default=0, help="pages per token and kv head (0: all)")
    ap.add_argument("--bits", type=int, choices=(4, 8), default=4)
    ap.add_argument("--keep", type=int, default=0, help="tokens that a sequence keeps, with 8 bits (0: all)")
    a = ap.parse_args()
    if a.bits == 8 and a.budget or a.bits == 4 and a.keep:
        ap.error("--budget is for 4 bits, --keep for 8")
    prompts = [int(p) for p in a.prompts.split(",")]
    size = dict(max_tokens=max(8, sum(prompts)), sequences=len(prompts), context=max(prompts) + a.steps)
    d = Decoder(bits=a.bits, keep=a.keep, **size)
    run(prompts, a.steps, a.budget, d)  # warm-up
    torch.cuda.synchronize()
    t = time.perf_counter()
    outs = run(prompts, a.steps, a.budget, d)
    torch.cuda.synchronize()
    t = time.perf_counter() - t
    whole = d if not a.keep else Decoder(bits=8, **size)
    dense = run(prompts, a.steps, 0, whole)
    off = float((outs[-1] - dense[-1]).norm() / dense[-1].norm())
    how = f"over {a.budget} pages: {off:.2e} from all" if a.budget else f"over {a.keep} tokens: {off:.2e} from all" if a.keep else "over all tokens"
    print(f"{len(prompts)} prompts of {prompts} tokens and {a.steps} steps in {t * 1e3:.1f} ms; last step {how}; "
          f"cache {d.cache.pages.numel() / 1e6:.1f} MB (16 bits: "
          f"{d.cache.pages.shape[1] * d.page_size * 4 * d.kv_heads * d.head_dim * len(d.qkv) / 1e6:.1f} MB)")
    if whole is not d:
        whole.close()
    d.close()


if __name__ == "__main__":
    main()
