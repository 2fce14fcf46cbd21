"""Forwards of one plan on streams that share a handle value follow one another."""
import threading

import pytest

from synth import workloads as W

pytestmark = pytest.mark.gpu

PER_THREAD = 2  # cudaStreamPerThread: one handle value, a stream in each thread


@pytest.mark.parametrize("T", [4, 200])
def test_per_thread_default_streams_of_two_threads(T):
    import torch

    from moe_expert_layer_sorted_gb300 import harness
    wl = W.WORKLOADS["tiny"]
    plan, _ = harness.build_plan(wl, max_tokens=256)
    xs = [torch.from_numpy(W.tokens(wl, 70 + i, 0, T)).cuda().view(torch.bfloat16) for i in range(6)]
    want, outs = ([torch.zeros_like(x) for x in xs] for _ in "ab")
    for x, y in zip(xs, want):
        plan.forward(0, x, y)
    torch.cuda.synchronize()
    turns = [threading.Semaphore(1), threading.Semaphore(0)]
    errors = []

    def work(t):
        try:
            for i in range(t, len(xs), 2):
                assert turns[t].acquire(timeout=60)
                plan.forward(0, xs[i], outs[i], stream=PER_THREAD)
                turns[1 - t].release()
        except BaseException as e:  # noqa: B036
            errors.append(e)
            turns[1 - t].release()

    threads = [threading.Thread(target=work, args=(t,)) for t in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not errors
    assert all(torch.equal(a.view(torch.int16), b.view(torch.int16)) for a, b in zip(outs, want))
    plan.close()
