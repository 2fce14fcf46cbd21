"""Calls of one cache handle on streams of their own: the ones that share its workspace follow
one another."""
import threading

import pytest
import torch

from test_gpu_kv_cache import BF, World

pytestmark = pytest.mark.gpu

PER_THREAD = 2  # cudaStreamPerThread: one handle value, a stream in each thread


def test_per_thread_default_streams_of_two_threads():
    """Attention whose items are cut between CTAs (partial results and counters in the
    workspace), from two threads that take turns."""
    w = World(128, 64, 64, BF, 2, [60000], seed=3).fill()
    qs = [w.rand(1, 1, 16, 128) for _ in range(6)]
    want = [torch.empty_like(q) for q in qs]
    for q, o in zip(qs, want):
        w.cache.attention(q, o, **w.batch)
    torch.cuda.synchronize()
    outs = [torch.zeros_like(q) for q in qs]
    torch.cuda.synchronize()
    turns = [threading.Semaphore(1), threading.Semaphore(0)]
    errors = []

    def work(t):
        try:
            for i in range(t, len(qs), 2):
                assert turns[t].acquire(timeout=60)
                w.cache.attention(qs[i], outs[i], stream=PER_THREAD, **w.batch)
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
    assert all(torch.equal(a, b) for a, b in zip(outs, want))


def test_calls_on_other_streams_beside_a_capture():
    """Asking for a stream's identity does not end the capture of another."""
    a, b = (World(128, 64, 64, BF, 2, [3000], seed=s).fill() for s in (4, 5))
    q = a.rand(1, 1, 16, 128)
    want, outs = [torch.empty_like(q) for _ in "ab"], [torch.zeros_like(q) for _ in "abcd"]
    for w, o in zip((a, b), want):
        w.cache.attention(q, o, **w.batch)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        a.cache.attention(q, outs[0], **a.batch)
        for s, o in zip(streams, outs[1:]):
            b.cache.attention(q, o, stream=s, **b.batch)
    g.replay()
    torch.cuda.synchronize()
    b.cache.attention(q, outs[3], **b.batch)
    assert torch.equal(outs[0], want[0]) and all(torch.equal(o, want[1]) for o in outs[1:])
