"""Eviction from sequences with more tokens than a CTA keeps at hand."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("batch,heads,n,budget,first,last", [(32, 8, 20000, 16384, 4, 256), (1, 1, 300000, 150001, 64, 1000),
                                                             (1, 2, 262160, 70000, 0, 0)])
def test_more_tokens_than_a_cta_holds(batch, heads, n, budget, first, last):
    """Many sequences of 20,000 tokens, and one of 300,000.  All codes of a step of 1, so that what moves is moved as it is."""
    from moe_expert_layer_sorted_gb300 import KVCache8
    D, P = 64, 64
    pages = -(-n // P)
    gen = torch.Generator(device="cuda").manual_seed(n)
    cache = KVCache8.allocate(batch * pages, kv_heads=heads, head_dim=D, page_size=P)
    table = torch.randperm(batch * pages, generator=gen, device="cuda").int().view(batch, pages)
    rows = [torch.randint(-127, 128, (batch, n, heads, D), generator=gen, device="cuda", dtype=torch.int16).bfloat16() for _ in range(2)]
    for x in rows:
        x[..., 5] = 127.0
    mass = torch.exp(2 * torch.randn(batch, heads, n, generator=gen, device="cuda"))
    mass[:, :, ::7] = mass[:, :, 3:4]  # ties
    lens = torch.full((batch,), n, dtype=torch.int32, device="cuda")
    lens[1::3] = n - 900
    lens[2::5] = budget
    cache.append(*rows, table=table, lens=torch.full_like(lens, n))
    paged = torch.zeros(batch, heads, pages * P, device="cuda")
    paged[:, :, :n] = mass
    cache.mass[0, table.long()] = paged.unflatten(2, (pages, P)).transpose(1, 2)
    kept = torch.empty(batch, heads, budget, dtype=torch.int32, device="cuda")
    cache.evict(kept, table=table, lens=lens, keep_first=first, keep_last=last)
    j = torch.arange(n, device="cuda")
    back = [torch.empty(batch, budget, heads, D, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    cache.read(*back, table=table, lens=lens.clamp_max(budget))
    now = cache.mass[0, table.long()].transpose(1, 2).flatten(2)
    for b, m in enumerate(lens.tolist()):
        rank = mass[b].clone()
        rank[:, (j < first) | (j >= m - last)] = float("inf")
        want = torch.sort(rank[:, :m], dim=1, descending=True, stable=True).indices[:, :budget].sort(1).values
        assert torch.equal(kept[b].long(), want), b
        for x, y in zip(rows, back):
            assert torch.equal(y[b], x[b].gather(0, want.T[..., None].expand(-1, -1, D))), b
        assert torch.equal(now[b, :, :budget], mass[b].gather(1, want))
        if m > budget:
            assert torch.equal(now[b, :, budget:n], mass[b, :, budget:])
