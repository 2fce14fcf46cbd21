"""Branches of the key/value cache's kernels that go by sizes: every instantiation of the
attention, more groups of rows than a CTA has threads, long tables, many kv heads, outputs of
the smallest alignment, the shared workspace on two streams."""
import math

import pytest
import torch

import kv_bounds
import kv_reference as ref
from test_gpu_kv_cache import BF, FP, World, starts_of

pytestmark = pytest.mark.gpu

EVERY = [(D, G, dtype) for D, G in ((64, 32), (64, 64), (128, 32), (128, 64), (128, 128)) for dtype in (BF, FP)]


def run(w, counts, q_heads, ragged=True):
    q = w.rand(sum(counts), q_heads, w.D)
    out, lse = torch.full_like(q, 9.0), torch.full(q.shape[:2], 9.0, device="cuda")
    w.cache.attention(q, out, lse=lse, starts=starts_of(counts), max_new=max(counts), **w.batch)
    at = 0
    for i, n in enumerate(counts):
        want = kv_bounds.attention(q[at:at + n], *w.values(i), kv_bounds.causal(n, w.lens[i]), 1 / math.sqrt(w.D), w.G)
        kv_bounds.check(out[at:at + n], lse[at:at + n], want, f"sequence {i}")
        at += n


@pytest.mark.parametrize("D,G,dtype", EVERY)
@pytest.mark.parametrize("per,counts", [(1, [1, 1, 1]), (5, [1, 1, 1]), (8, [2, 1, 1]), (3, [4, 2, 3]), (16, [1, 2, 1]),
                                        (4, [40, 9, 1])])
def test_every_instantiation(D, G, dtype, per, counts):
    """1 to 8, 9 to 16, 17 to 32 columns, and the prompt kernel."""
    run(World(D, G, 32, dtype, 2, [777, 40, 130], seed=per).fill(), counts, 2 * per)


@pytest.mark.parametrize("n", [1, 2, 3, 4, 5, 9])
@pytest.mark.parametrize("D,G,dtype", [(128, 64, BF), (64, 32, FP)])
def test_writes_of_a_few_rows_and_one_write_are_the_same_bytes(D, G, dtype, n):
    a, b = (World(D, G, 32, dtype, 2, [75, 40, 3], seed=5) for _ in "ab")
    a.fill()
    for have in range(n, 75 + n, n):
        lens = torch.tensor([min(have, L) for L in a.lens], dtype=torch.int32, device="cuda")
        counts = [max(min(have, L) - (have - n), 0) for L in a.lens]
        rows = [torch.cat([x[i][have - n:have - n + c] for i, c in enumerate(counts)]) for x in (b.k, b.v)]
        b.cache.append(*rows, table=b.table, lens=lens, starts=starts_of(counts), max_new=n)
    assert torch.equal(a.cache.pages, b.cache.pages)
    assert torch.equal(a.cache.bounds.view(torch.int16), b.cache.bounds.view(torch.int16))


def test_more_sequences_than_threads():
    g = torch.Generator().manual_seed(0)
    lens = torch.randint(1, 60, (500,), generator=g).tolist()
    run(World(128, 64, 16, BF, 2, lens, seed=8).fill(), [1] * 500, 8)
    counts = [2 if i % 3 == 0 and n > 1 else 1 for i, n in enumerate(lens)]
    run(World(64, 32, 16, FP, 1, lens, seed=9).fill(), counts, 4)


@pytest.mark.parametrize("dtype,per", [(BF, 4), (FP, 12)])
def test_chosen_pages_of_more_rows_than_threads(dtype, per):
    """With rows of nobody between them, which keep what they held."""
    w = World(128, 64, 16, dtype, 2, [700, 500], seed=per).fill()
    counts, budget = [500, 170], 5
    q = w.rand(720, 2 * per, 128)
    starts = torch.tensor([20, 520, 690], dtype=torch.int32, device="cuda")
    at = dict(starts=starts, max_new=500, **w.batch)
    pages = torch.full((720, 2, budget), -7, dtype=torch.int32, device="cuda")
    w.cache.select(q, pages, **at)
    out, lse = torch.full_like(q, 9.0), torch.full((720, 2 * per), 9.0, device="cuda")
    w.cache.attention(q, out, lse=lse, pages=pages, **at)
    for rows in (slice(0, 20), slice(690, 720)):
        assert (pages[rows] == -7).all() and (out[rows] == 9).all() and (lse[rows] == 9).all()
    for i, (first, n) in enumerate(((20, 500), (520, 170))):
        L = w.lens[i]
        t = torch.arange(L, device="cuda")
        k, v = w.values(i)
        ends = w.cache.bounds[0][w.table[i].long().clamp_min(0)].cpu()
        for j in range(0, n, 61):
            for h in range(2):
                mine = pages[first + j, h].cpu().tolist()
                heads = slice(h * per, (h + 1) * per)
                assert mine == ref.select(q[first + j, heads].cpu(), ends[:, h, 0], ends[:, h, 1], (L - n + j) // 16 + 1, budget, 1, 1)
                seen = torch.isin(t // 16, torch.tensor(mine, device="cuda")) & (t <= L - n + j)
                want = kv_bounds.attention(q[first + j:first + j + 1, heads], k[:, h:h + 1], v[:, h:h + 1], seen[None], 1 / math.sqrt(128), 64)
                kv_bounds.check(out[first + j:first + j + 1, heads], lse[first + j:first + j + 1, heads], want, f"{i} {j} {h}")


@pytest.mark.parametrize("pages,heads", [(5000, 1), (4097, 3), (600, 17), (4096, 2), (513, 20), (5000, 33)])
def test_selection_over_long_tables_and_many_heads(pages, heads):
    from moe_expert_layer_sorted_gb300 import KVCache
    g = torch.Generator(device="cuda").manual_seed(pages + heads)
    c = KVCache.allocate(pages, kv_heads=heads, head_dim=64, page_size=16, group_size=32)
    hi = torch.randn(1, pages, heads, 64, generator=g, device="cuda").to(BF)
    c.bounds[:, :, :, 0], c.bounds[:, :, :, 1] = hi, hi - torch.rand(hi.shape, generator=g, device="cuda").to(BF)
    table = torch.randperm(pages, generator=g, device="cuda").int().expand(3, pages).contiguous()
    lens = torch.tensor([16 * pages - 5, 16 * (pages // 2), 16 * 40], dtype=torch.int32, device="cuda")
    q = torch.randn(3, 1, 2 * heads, 64, generator=g, device="cuda").to(BF)
    for budget in (4, 65):
        out = torch.empty(3, heads, budget, dtype=torch.int32, device="cuda")
        c.select(q, out, table=table, lens=lens)
        ends = c.bounds[0][table[0].long()].cpu()
        for i in range(3):
            for h in {0, heads // 2, heads - 1, min(16, heads - 1)}:
                n = (int(lens[i]) - 1) // 16 + 1
                assert out[i, h].tolist() == ref.select(q[i, 0, 2 * h:2 * h + 2].cpu(), ends[:, h, 0], ends[:, h, 1], n, budget, 1, 1)


@pytest.mark.parametrize("D,G,dtype", [(128, 64, BF), (64, 32, FP)])
@pytest.mark.parametrize("lens", [[300], [9000]])
def test_prompt_outputs_of_the_smallest_alignment(D, G, dtype, lens):
    w = World(D, G, 32, dtype, 2, lens, seed=1).fill()
    q = w.rand(1, 70, 6, D)
    want = torch.empty_like(q)
    w.cache.attention(q, want, **w.batch)
    room = torch.full((70 * (6 * D + 8) + 8,), 3.0, dtype=dtype, device="cuda")
    out = room[8:].as_strided((1, 70, 6, D), (0, 6 * D + 8, D, 1), 8)  # 16 bytes past a multiple of 32
    assert out.data_ptr() % 32 == 16
    w.cache.attention(q, out, **w.batch)
    assert torch.equal(out, want)
    kept = torch.ones(room.shape, dtype=torch.bool, device="cuda")
    kept.as_strided((1, 70, 6, D), (0, 6 * D + 8, D, 1), 8).fill_(False)
    assert (room[kept] == 3).all()


def test_the_workspace_on_two_streams_in_turn():
    """Scores of long tables, parts of prompts that are cut into stretches and of single tokens
    that are cut between CTAs lie in one workspace."""
    w = World(128, 64, 16, BF, 2, [16 * 700], seed=2).fill()
    q, prompt = w.rand(1, 1, 16, 128), w.rand(1, 40, 16, 128)

    def calls(stream):
        pages = torch.full((1, 2, 33), -7, dtype=torch.int32, device="cuda")
        a, b = torch.zeros_like(q), torch.zeros_like(prompt)
        torch.cuda.synchronize()
        return [(pages, lambda: w.cache.select(q, pages, stream=stream, **w.batch)),
                (b, lambda: w.cache.attention(prompt, b, stream=stream, **w.batch)),
                (a, lambda: w.cache.attention(q, a, stream=stream, **w.batch))]

    want = calls(None)
    for _, f in want:
        f()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for order in range(3):
        each = [calls(s) for s in streams]
        for i in range(12):  # the streams in turn, each call beside another kind
            out, f = each[i % 2][(i // 2 + order * (i % 2)) % 3]
            f()
        torch.cuda.synchronize()
        for side in each:
            for (got, _), (ok, _) in zip(side, want):
                assert torch.equal(got, ok)
