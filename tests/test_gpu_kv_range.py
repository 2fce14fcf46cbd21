"""Attention over the 4-bit cache where sizes differ by many powers of two: each row's result
is bounded by what that row sees and weighs (kv_bounds.py)."""
import math

import pytest
import torch

import kv_bounds
from test_gpu_kv_cache import BF, FP, World

pytestmark = pytest.mark.gpu


def run(w, n, q=None, per=4, scale=None, causal=True, what=""):
    """n rows of every sequence of w."""
    q = w.rand(len(w.lens), n, per * w.heads, w.D) if q is None else q
    out, lse = torch.full_like(q, 9.0), torch.full((len(w.lens) * n, q.shape[2]), 9.0, device="cuda")
    w.cache.attention(q, out, lse=lse, scale=scale, causal=causal, **w.batch)
    for i, L in enumerate(w.lens):
        seen = kv_bounds.causal(n, L) if causal else torch.ones(n, L, dtype=torch.bool, device="cuda")
        want = kv_bounds.attention(q[i], *w.values(i), seen, 1 / math.sqrt(w.D) if scale is None else scale)
        kv_bounds.check(out[i], lse[i * n:(i + 1) * n], want, f"{what} sequence {i}")


@pytest.mark.parametrize("n", [1, 3, 80])
@pytest.mark.parametrize("scale", [None, 6.0])
def test_queries_up_to_the_types_largest(n, scale):
    """Queries of 2^118 to 2^127 over keys so small that the scores are ordinary."""
    w = World(128, 64, 32, BF, 2, [150, 150], seed=n)
    w.k[0] = (w.k[0].float() * 2.0 ** -121).to(BF)
    w.k[1] = (w.k[1].float() * 2.0 ** -117).to(BF)
    w.fill()
    q = w.rand(2, n, 8, 128).float().clamp(-3.9, 3.9)
    q[0] *= 2.0 ** (121 if scale is None else 119)
    q[1] *= 2.0 ** (117 if scale is None else 115)
    q[0, 0, 0, 5] = 2.0 ** (126 if scale is None else 122)
    run(w, n, q.to(BF), scale=scale)
