"""Attention over the 8-bit cache with queries and keys of far sizes, and what it adds to the mass of its tokens."""
import pytest

from test_gpu_kv8 import BF, World, run_attention

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("rows", [1, 40])
@pytest.mark.parametrize("up", [100, 122])
def test_large_queries_over_small_keys(rows, up):
    """Their products are of ordinary size, at every step of the way."""
    w = World(64, 16, BF, 2, [300], seed=rows)
    w.k[0] = (w.k[0].double() * 2.0 ** -up).to(BF)
    w.fill()
    q = (w.rand(rows, 4, 64).double() * 2.0 ** up).to(BF)
    run_attention(w, [rows], 4, q=q, weigh=True)
