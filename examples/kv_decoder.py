"""A small decoder whose attention keeps its keys and values in 4 bits and whose
feed-forward layers are sparse MoE layers, run as a server would: prompts of different
lengths first, in one ragged batch, then single tokens, over the whole context or over the
pages that the cache's bounds choose.

    python examples/kv_decoder.py [--steps 16] [--prompts 300,41,128] [--budget 0]

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

from moe_expert_layer_sorted_gb300 import KVCache, harness  # noqa: E402
from synth import workloads as W  # noqa: E402


def norm(x):
    """Root-mean-square norm of the fp32 residual stream, in bf16."""
    return (x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6)).to(torch.bfloat16)


class Decoder:
    """`layers` times: attention over the 4-bit cache, then the MoE layer; fp32 residual."""

    def __init__(self, layers=2, q_heads=8, kv_heads=2, head_dim=64, max_tokens=1024, sequences=4, context=2048, page_size=16,
                 seed=0):
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
        self.cache = KVCache.allocate(sequences * per_seq, kv_heads=kv_heads, head_dim=head_dim, page_size=page_size,
                                      group_size=32, layers=layers)
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
            self.cache.attention(q, o, pages=pages, layer=layer, **batch)
            x = x + (o.view(n, -1) @ wout).float()
            h = norm(x)
            y, mixed = torch.empty_like(h), torch.empty_like(h)
            # the MoE layer with the residual added in its combine; the example keeps the stream in fp32
            self.plan.forward_residual(0, h, y, x, mixed)
            x = x + y.float()
        return x


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
        lens = lens + 1
        outs.append(d.forward(inputs(len(prompts), d.wl.hidden, seed + 1 + i), lens, budget=budget))
    return outs


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--steps", type=int, default=16)
    ap.add_argument("--prompts", default="300,41,128")
    ap.add_argument("--budget", type=int, default=0, help="pages per token and kv head (0: all)")
    a = ap.parse_args()
    prompts = [int(p) for p in a.prompts.split(",")]
    d = Decoder(max_tokens=max(8, sum(prompts)), sequences=len(prompts), context=max(prompts) + a.steps)
    run(prompts, a.steps, a.budget, d)  # warm-up
    torch.cuda.synchronize()
    t = time.perf_counter()
    outs = run(prompts, a.steps, a.budget, d)
    torch.cuda.synchronize()
    t = time.perf_counter() - t
    dense = run(prompts, a.steps, 0, d)
    off = float((outs[-1] - dense[-1]).norm() / dense[-1].norm())
    print(f"{len(prompts)} prompts of {prompts} tokens and {a.steps} steps in {t * 1e3:.1f} ms; last step "
          f"{'over all pages' if not a.budget else f'over {a.budget} pages: {off:.2e} from all'}; "
          f"cache {d.cache.pages.numel() / 1e6:.1f} MB (16 bits: "
          f"{d.cache.pages.shape[1] * d.page_size * 4 * d.kv_heads * d.head_dim * len(d.qkv) / 1e6:.1f} MB)")
    d.close()


if __name__ == "__main__":
    main()
