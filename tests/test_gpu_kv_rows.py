"""Rows that are no sequence's tokens, and rows whose scores are very low."""
import math

import pytest
import torch

import kv_bounds
from test_gpu_kv_cache import BF, FP, World

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("D,G,P,dtype", [(128, 64, 16, BF), (64, 32, 32, FP)])
@pytest.mark.parametrize("n", [3, 7, 90])
@pytest.mark.parametrize("chosen", [False, True])
def test_rows_before_a_sequence_attend_to_nothing_without_causal_mask_too(D, G, P, dtype, n, chosen):
    w = World(D, G, P, dtype, 2, [2, n - 1, 40, 130], seed=n).fill()
    q = w.rand(4, n, 4, D)
    out, lse = torch.full_like(q, 9.0), torch.full((4 * n, 4), 9.0, device="cuda")
    pages = torch.arange(9, dtype=torch.int32, device="cuda").expand(4 * n, 2, 9).contiguous() if chosen else None
    w.cache.attention(q, out, lse=lse, causal=False, pages=pages, **w.batch)
    for i, L in enumerate(w.lens):
        seen = (torch.arange(L - n, L, device="cuda") >= 0)[:, None].expand(n, L)
        kv_bounds.check(out[i], lse[i * n:(i + 1) * n], kv_bounds.attention(q[i], *w.values(i), seen, 1 / math.sqrt(D), G))
