"""The example decoder (examples/kv_decoder.py): ragged prompts, steps over all pages and
over chosen ones, beside the MoE layer."""
import os
import sys

import pytest

from conftest import ROOT

pytestmark = pytest.mark.gpu
sys.path.insert(0, os.path.join(ROOT, "examples"))


@pytest.fixture(scope="module")
def decoder():
    import kv_decoder
    d = kv_decoder.Decoder(max_tokens=600, sequences=3, context=512)
    yield d
    d.close()


def typical(got, want):
    """The middle sequence's relative difference.  Rows are a few bf16 roundings (2^-8) apart in
    each of two layers; one whose experts or stored codes tip over differs altogether."""
    return float(((got - want).norm(dim=-1) / want.norm(dim=-1)).median())


def test_steps_after_prompts_are_the_longer_prompts(decoder):
    """A prompt and one step give what the prompt with that token gives: the same keys and
    values are stored, and the two attention kernels agree within their roundings."""
    import kv_decoder
    import torch
    prompts = [200, 41, 130]
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


def test_a_budget_of_all_pages_is_the_whole_context(decoder):
    import kv_decoder
    prompts = [100, 41, 63]
    dense = kv_decoder.run(prompts, 3, decoder=decoder)
    all_pages = kv_decoder.run(prompts, 3, budget=7, decoder=decoder)
    some = kv_decoder.run(prompts, 3, budget=3, decoder=decoder)
    for a, b, c in zip(dense, all_pages, some):
        assert typical(b, a) < 0.05
        assert typical(c, a) < 1.0
    assert not (dense[-1] == some[-1]).all()
