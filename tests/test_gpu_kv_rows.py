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


@pytest.mark.parametrize("n", [1, 4, 90])
@pytest.mark.parametrize("length", [200, 5000])
@pytest.mark.parametrize("size", [2.0 ** 11, 2.0 ** 13, 2.0 ** 16, -2.0 ** 13])
def test_scores_of_millions_and_more(n, length, size):
    """Where a score's last place is above one: a row is the mean of the tokens that score the
    same and more than all others."""
    w = World(128, 64, 64, BF, 2, [length], seed=n)
    u = w.rand(2, 128).sign()
    w.k[0].copy_((w.k[0].float().clamp(-1, 1) * 0.3 * abs(size)).to(BF))
    best = torch.arange(7, length - n, 31, device="cuda")
    w.k[0][best] = u * size
    w.fill()
    q = (u * abs(size)).expand(1, n, 2, 128).to(BF) * (1 if size > 0 else -1)
    out, lse = torch.full((1, n, 2, 128), 9.0, dtype=BF, device="cuda"), torch.empty(n, 2, device="cuda")
    w.cache.attention(q, out, lse=lse, **w.batch)
    k, v = w.values(0)
    score = (q[0, 0].double() * k[best[0]]).sum(-1) / math.sqrt(128)
    assert (score > 1e6).all()
    want = v[best].mean(0)
    assert ((out[0].double() - want).abs() <= 2.0 ** -8 * want.abs() + 2.0 ** -8).all()
    assert ((lse.double() / score - 1).abs() < 2.0 ** -11).all()


@pytest.mark.parametrize("n", [1, 4, 90])
@pytest.mark.parametrize("size", [2.0 ** 12, 2.0 ** 15, 2.0 ** 40])
@pytest.mark.parametrize("sign", [1, -1])
def test_equal_scores_of_millions_and_more(n, size, sign):
    w = World(128, 64, 64, BF, 1, [3000], seed=n)
    w.k[0].copy_((w.k[0][:1].float() * size).to(BF).expand(3000, 1, 128))
    w.fill()
    q = (w.k[0][:1].float() * sign).to(BF).expand(1, n, 4, 128)
    out = torch.full((1, n, 4, 128), 9.0, dtype=BF, device="cuda")
    w.cache.attention(q, out, **w.batch)
    _, v = w.values(0)
    for i in range(n):
        want = v[:3000 - n + i + 1].mean(0)
        assert ((out[0, i].double() - want).abs() <= 2.0 ** -8 * want.abs() + 2.0 ** -9).all()


@pytest.mark.parametrize("n", [1, 4, 90])
@pytest.mark.parametrize("length", [200, 5000])
def test_scores_near_the_lowest_fp32(n, length):
    """Every token scores the same, some -10^36: the row is the mean of what it sees."""
    w = World(128, 64, 64, BF, 1, [length], seed=n)
    w.k[0].copy_((w.k[0][:1].float() * 2.0 ** 64).to(BF).expand(length, 1, 128))
    w.fill()
    q = (-w.k[0][:1].float() * 2.0 ** -10).to(BF).expand(1, n, 4, 128)
    out, lse = torch.full((1, n, 4, 128), 9.0, dtype=BF, device="cuda"), torch.empty(n, 4, device="cuda")
    w.cache.attention(q, out, lse=lse, **w.batch)
    k, v = w.values(0)
    score = float((q[0, 0, 0].double() @ k[0, 0])) / math.sqrt(128)
    assert -3e38 < score < -1e34
    for i in range(n):
        want = v[:length - n + i + 1].mean(0)
        assert ((out[0, i].double() - want).abs() <= 2.0 ** -8 * want.abs() + 2.0 ** -9).all()
    assert ((lse.double() / score - 1).abs() < 2.0 ** -16).all()
