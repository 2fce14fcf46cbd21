"""The failure path of the cache's attention without a fault: a bounded wait runs out, the
kernel ends by itself, the next call says so, and what follows is right."""
import pytest
import torch

from test_gpu_kv_cache import BF, FP, World

pytestmark = pytest.mark.gpu


def setup(kind):
    w = World(128, 64, 64, BF if kind == "prompt" else FP, 2, [20000, 300] if kind == "split" else [3000, 300], seed=3).fill()
    q = w.rand(2, 100 if kind == "prompt" else 1, 8, 128)
    want = torch.empty_like(q)
    w.cache.attention(q, want, **w.batch)
    return w, q, want


@pytest.mark.parametrize("kind", ["split", "single", "prompt"])
def test_reported_by_the_next_call_and_nothing_stays(kind):
    from moe_expert_layer_sorted_gb300 import MoeError
    w, q, want = setup(kind)
    out = torch.empty_like(q)
    calls = [lambda: w.cache.attention(q, out, **w.batch), w.cache.check,
             lambda: w.cache.read(w.k[0][None, -1:], w.v[0][None, -1:], table=w.table[:1], lens=w.lens_t[:1], layer=0)]
    for call in calls:
        w.cache.debug_fail_next_attention()
        w.cache.attention(q, out, **w.batch)
        torch.cuda.synchronize()
        with pytest.raises(MoeError) as e:
            call()
        assert e.value.status == 4
        for _ in range(3):
            out.zero_()
            w.cache.attention(q, out, **w.batch)
            assert torch.equal(out, want)
        w.cache.check()


@pytest.mark.parametrize("kind", ["split", "prompt"])
def test_a_graph_replayed_after_a_failure_is_right(kind):
    """No host call stands between the failure and the replays."""
    from moe_expert_layer_sorted_gb300 import MoeError
    w, q, want = setup(kind)
    torch.cuda.synchronize()
    out, bad = torch.empty_like(q), torch.empty_like(q)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        w.cache.attention(q, out, **w.batch)
    w.cache.debug_fail_next_attention()
    w.cache.attention(q, bad, **w.batch)
    for _ in range(3):
        torch.cuda.synchronize()
        out.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)
    with pytest.raises(MoeError, match="gave up"):
        w.cache.check()
    g.replay()
    torch.cuda.synchronize()
    w.cache.check()
