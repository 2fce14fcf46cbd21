"""The example decoder (examples/kv_decoder.py) over the 8-bit cache: prompts, steps, eviction, beside the MoE layer."""
import os
import sys

import pytest

from conftest import ROOT

pytestmark = pytest.mark.gpu
sys.path.insert(0, os.path.join(ROOT, "examples"))


def made(**kw):
    import kv_decoder
    return kv_decoder.Decoder(max_tokens=600, sequences=3, context=512, bits=8, **kw)


def typical(got, want):
    """The middle sequence's relative difference.  Rows are a few bf16 roundings (2^-8) apart in
    each of two layers; one whose experts tip over differs altogether."""
    return float(((got - want).norm(dim=-1) / want.norm(dim=-1)).median())


def test_steps_after_prompts_are_the_longer_prompts():
    import kv_decoder
    import torch
    decoder, prompts = made(), [200, 41, 130]
    outs = kv_decoder.run(prompts, 1, decoder=decoder)
    hidden = decoder.wl.hidden
    first, more = kv_decoder.inputs(sum(prompts), hidden, 1), kv_decoder.inputs(3, hidden, 2)
    rows, at = [], 0
    for i, n in enumerate(prompts):
        rows += [first[at:at + n], more[i:i + 1]]
        at += n
    lens = torch.tensor([n + 1 for n in prompts], dtype=torch.int32, device="cuda")
    starts = torch.zeros(4, dtype=torch.int32, device="cuda")
    starts[1:] = torch.cumsum(lens, 0)
    x = decoder.forward(torch.cat(rows), lens, starts, max(prompts) + 1)
    ends = starts[1:].long() - 1
    for got, want in ((outs[0], x[ends - 1]), (outs[1], x[ends])):
        assert torch.isfinite(got).all()
        assert typical(got, want) < 0.05
    decoder.close()


def test_a_cache_at_a_budget():
    """More tokens than there are: the same bits as without; fewer: other results, all finite, and the cache's
    lengths stay at the budget."""
    import kv_decoder
    import torch
    prompts = [100, 41, 63]
    runs = {}
    for keep in (0, 400, 32):
        d = made(keep=keep)
        runs[keep] = kv_decoder.run(prompts, 3, decoder=d)
        if keep == 32:
            lens = torch.tensor([100, 20, 33], dtype=torch.int32, device="cuda")
            assert d.evict(lens).tolist() == [32, 20, 32]
        d.close()
    for a, b, c in zip(runs[0], runs[400], runs[32]):
        assert torch.equal(a, b)
        assert torch.isfinite(c).all() and typical(c, a) < 1.5
    assert torch.equal(runs[0][0], runs[32][0]) and not torch.equal(runs[0][-1], runs[32][-1])
