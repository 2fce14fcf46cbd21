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
        want = kv_bounds.attention(q[i], *w.values(i), seen, 1 / math.sqrt(w.D) if scale is None else scale, w.G)
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


SHAPES = [(128, 64, 64, BF), (64, 32, 16, BF), (128, 32, 32, FP), (128, 128, 64, BF)]


def times(x, factor, dtype):
    return (x.float() * factor).clamp(-torch.finfo(dtype).max, torch.finfo(dtype).max).to(dtype)


@pytest.mark.parametrize("D,G,P,dtype", SHAPES)
@pytest.mark.parametrize("n", [2, 5, 80, 200])
def test_a_huge_value_that_only_the_last_row_sees(D, G, P, dtype, n):
    """The rows before it are what they are without it."""
    w = World(D, G, P, dtype, 2, [n, 333, 1500], seed=n)
    for v in w.v:
        if dtype == FP:
            v.copy_(times(v, 2.0 ** -12, dtype))
        v[-1] = times(v[-1], 1e9 if dtype == BF else 2.0 ** 27, dtype)
    w.fill()
    run(w, n)


@pytest.mark.parametrize("D,G,P,dtype", SHAPES)
@pytest.mark.parametrize("n", [1, 3, 80])
@pytest.mark.parametrize("at", [0, 5, 40])
def test_a_huge_value_of_no_weight(D, G, P, dtype, n, at):
    """A token that every row sees, its score some 100 below the others'."""
    w = World(D, G, P, dtype, 2, [n + at + 1, 700], seed=n + at)
    q = w.rand(2, n, 8, D)
    q[..., 0] = 8.0
    for i in range(2):
        if dtype == FP:
            w.v[i].copy_(times(w.v[i], 2.0 ** -12, dtype))
        w.k[i][at, :, 0] = -100 * math.sqrt(D) / 8
        w.v[i][at] = times(w.v[i][at], 1e9 if dtype == BF else 2.0 ** 27, dtype)
    run(w.fill(), n, q)


@pytest.mark.parametrize("D,G,P,dtype", SHAPES)
@pytest.mark.parametrize("n", [1, 3, 80])
@pytest.mark.parametrize("at", [0, 7, 300])
@pytest.mark.parametrize("size", [0.0, 2.0 ** -30, 2.0 ** -9])
def test_a_token_of_nearly_all_the_weight_and_hardly_any_value(D, G, P, dtype, n, at, size):
    """What is left of the weights, some 2^-30, carries the result."""
    w = World(D, G, P, dtype, 2, [400 + n, 700], seed=n + at)
    q = w.rand(2, n, 8, D)
    q[..., 0] = 8.0
    for i in range(2):
        w.k[i][at, :, 0] = 20 * math.sqrt(D) / 8
        w.v[i][at] = times(w.v[i][at], size, dtype)
    run(w.fill(), n, q)


@pytest.mark.parametrize("D,G,P,dtype", SHAPES)
@pytest.mark.parametrize("n", [1, 3, 80])
@pytest.mark.parametrize("kind", ["tokens", "blocks", "up", "down", "zeros"])
def test_values_of_all_sizes(D, G, P, dtype, n, kind):
    w = World(D, G, P, dtype, 2, [n, 333, 2100], seed=n)
    most = 40 if dtype == BF else 10
    for v in w.v:
        L = len(v)
        t = torch.arange(L, device="cuda")
        e = torch.randint(-most, most + 1, (L, 2, 1), generator=w.g, device="cuda").float()
        if kind == "blocks":  # runs of 150 tokens
            e = e[(t // 150) * 150]
        elif kind in ("up", "down"):  # first tokens of another size
            e = torch.where(t[:, None, None] < 20, -most if kind == "up" else most, 0).float()
        v.copy_(times(v, torch.exp2(e), dtype))
        if kind == "zeros":
            v[::3] = 0
            v[100:400] = 0
    w.fill()
    run(w, n)
    run(w, n, scale=0.0)


@pytest.mark.parametrize("n", [1, 4, 60])
def test_parts_whose_values_are_far_apart(n):
    """One value near the type's largest among many parts of ordinary, tiny or zero values: every
    part keeps its share of the weights."""
    for size in (1.0, 2.0 ** -60, 0.0):
        w = World(128, 64, 64, BF, 2, [6000, 900, 70], seed=n)
        for i, v in enumerate(w.v):
            v.copy_(times(v, size, BF))
            v[3 + 2 * i] = torch.where(v[3 + 2 * i] < 0, -0.9, 0.9).to(BF) * torch.finfo(BF).max
        w.fill()
        run(w, n, scale=0.02, what=f"size {size}")


@pytest.mark.parametrize("D,G,P,dtype", SHAPES[:3])
@pytest.mark.parametrize("n", [1, 3, 80])
def test_groups_of_channels_far_apart(D, G, P, dtype, n):
    """Groups 2^16 apart, in every token or in some of any weight."""
    w = World(D, G, P, dtype, 2, [n + 300, 700], seed=n)
    for i, v in enumerate(w.v):
        v[:: 1 if i else 7, :, :G] = times(v[:: 1 if i else 7, :, :G], 2.0 ** -16, dtype)
    run(w.fill(), n)


@pytest.mark.parametrize("D,G,P,dtype", SHAPES)
@pytest.mark.parametrize("n", [1, 3, 40])
@pytest.mark.parametrize("above", [20, 27, 34])
def test_all_the_weight_on_tokens_without_values(D, G, P, dtype, n, above):
    """Half of the tokens have no values, one of them scores `above` more than any other token;
    what the others weigh, down to 2^-50, carries the result."""
    w = World(D, G, P, dtype, 2, [n + 3, n + 17, 200, 1000], seed=n + above)
    q = (0.3 * w.rand(4, n, 8, D).float()).to(dtype)
    q[..., 0] = 8.0
    for k, v in zip(w.k, w.v):
        k[:, :, 0] *= 0.1
        k[len(k) // 3, :, 0] = above * math.sqrt(D) / 8
        v[torch.arange(len(v), device="cuda") % 2 == len(v) // 3 % 2] = 0
        if dtype == FP:  # so that the results are above fp16's smallest
            v.copy_(times(v, 2.0 ** 12, dtype))
    run(w.fill(), n, q)
