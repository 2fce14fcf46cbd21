"""The 4-bit key/value cache on the GPU: format, writes, reads, attention and page selection
against the plain implementation, over head layouts, lengths, masks and strides where they
can go wrong."""
import math

import numpy as np
import pytest
import torch

import kv_reference as ref

pytestmark = pytest.mark.gpu

BF, FP = torch.bfloat16, torch.float16
GEOMETRY = [(64, 32, 16, BF), (64, 64, 64, FP), (128, 32, 32, FP), (128, 64, 64, BF), (128, 128, 256, BF), (128, 64, 128, FP)]


class World:
    """Sequences with known keys and values in a cache whose free memory is NaN."""

    def __init__(self, D, G, P, dtype, heads, lens, seed=0, spare=3, layers=1, layer=0):
        from moe_expert_layer_sorted_gb300 import KVCache
        self.D, self.G, self.P, self.dtype, self.heads, self.lens, self.layer = D, G, P, dtype, heads, list(lens), layer
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.g = g
        need = [-(-n // P) for n in lens]
        self.cols = max(need + [1])
        total = sum(need) + spare
        self.cache = KVCache.allocate(total, kv_heads=heads, head_dim=D, page_size=P, group_size=G, dtype=dtype, layers=layers)
        self.cache.pages.fill_(0xFF)  # params of all ones: NaN
        self.cache.bounds.fill_(math.nan)
        ids = torch.randperm(total, generator=g, device="cuda").int()
        self.table = torch.full((len(lens), self.cols), -1, dtype=torch.int32, device="cuda")
        at = 0
        for i, n in enumerate(need):
            self.table[i, :n] = ids[at:at + n]
            at += n
        self.lens_t = torch.tensor(self.lens, dtype=torch.int32, device="cuda")
        self.k = [self.rand(n, heads, D) * torch.exp(0.5 * torch.randn(heads, D, generator=g, device="cuda")).to(dtype) for n in lens]
        self.v = [self.rand(n, heads, D) for n in lens]

    def rand(self, *shape):
        return torch.randn(*shape, generator=self.g, device="cuda").to(self.dtype)

    def fill(self, upto=None):
        for i, n in enumerate(self.lens):
            n = n if upto is None else min(n, upto[i])
            if n:
                self.cache.append(self.k[i][None, :n], self.v[i][None, :n], table=self.table[i:i + 1], layer=self.layer,
                                  lens=torch.tensor([n], dtype=torch.int32, device="cuda"))
        return self

    def values(self, i):
        return ref.values(self.k[i], self.G), ref.values(self.v[i], self.G)

    @property
    def batch(self):
        return dict(table=self.table, lens=self.lens_t, layer=self.layer)


def starts_of(counts):
    return torch.tensor(np.concatenate([[0], np.cumsum(counts)]), dtype=torch.int32, device="cuda")


def same_bits(a, b):
    """Equal values, NaN where NaN."""
    return torch.equal(torch.isnan(a), torch.isnan(b)) and torch.equal(a.nan_to_num(7.0), b.nan_to_num(7.0))


def check(out, want, tol, what=""):
    d = (out.double() - want).abs()
    assert torch.isfinite(out).all(), what
    assert (d <= tol).all(), f"{what}: {float((d / tol).max())} of the bound"
    n = float(want.norm())
    if n:  # three independent roundings of at most a unit each
        assert float(d.norm()) <= 3.5 * ref.UNIT[out.dtype] * n + 1e-4 * n, what


# ------------------------------------------------------------------------ write and read

@pytest.mark.parametrize("D,G,P,dtype", GEOMETRY)
def test_layout_and_codes(D, G, P, dtype):
    w = World(D, G, P, dtype, 2, [P + 19]).fill()
    for pos0 in range(0, P + 19, 16):
        page, blk = int(w.table[0, pos0 // P]), pos0 % P // 16
        for h in range(2):
            ku, vu, kp, vp = ref.decode_block(w.cache.pages[0, page, h, blk].cpu().numpy(), D, G, dtype)
            for codes, par, x in ((ku, kp, w.k[0]), (vu, vp, w.v[0])):
                x = x[pos0:pos0 + 16, h].cpu()
                u, s, c = ref.quantise(x, G)
                assert np.array_equal(codes[:len(x)], u.numpy())
                assert torch.equal(par[:len(x), :, 0], s) and torch.equal(par[:len(x), :, 1], c)


@pytest.mark.parametrize("D,G,P,dtype", GEOMETRY)
def test_append_in_pieces_then_read(D, G, P, dtype):
    """A prompt, then single tokens, then a few: what is read is what was stored."""
    lens = [P + 23, 3, 70]
    w = World(D, G, P, dtype, 3, lens)
    have = [P + 17, 1, 2 * 16]
    w.fill(have)
    while have != lens:
        n = 1 if sum(have) % 3 else 2
        idx = [i for i in range(3) if have[i] < lens[i]]
        step = [min(n, lens[i] - have[i]) for i in idx]
        for i, m in zip(idx, step):
            have[i] += m
        k = torch.cat([w.k[i][have[i] - m:have[i]] for i, m in zip(idx, step)])
        v = torch.cat([w.v[i][have[i] - m:have[i]] for i, m in zip(idx, step)])
        w.cache.append(k, v, table=w.table[idx], starts=starts_of(step), max_new=2,
                       lens=torch.tensor([have[i] for i in idx], dtype=torch.int32, device="cuda"))
    k, v = (torch.full((sum(lens), 3, D), 5.0, dtype=dtype, device="cuda") for _ in range(2))
    w.cache.read(k, v, starts=starts_of(lens), max_new=max(lens), **w.batch)
    at = 0
    for i, n in enumerate(lens):
        kx, vx = w.values(i)
        assert same_bits(k[at:at + n], kx.to(dtype)) and same_bits(v[at:at + n], vx.to(dtype))
        at += n
        for j in range(-(-n // P)):  # the bounds are those of the page's stored keys
            rows = kx[j * P:(j + 1) * P].float().to(dtype)
            ends = w.cache.bounds[0, int(w.table[i, j])]
            assert torch.equal(ends[:, 0], rows.amax(0)) and torch.equal(ends[:, 1], rows.amin(0))


def test_pieces_and_one_write_are_the_same_bytes():
    a, b = World(128, 64, 32, BF, 2, [77]), World(128, 64, 32, BF, 2, [77])
    a.fill()
    for n in range(1, 78):
        b.cache.append(b.k[0][None, n - 1:n], b.v[0][None, n - 1:n], table=b.table,
                       lens=torch.tensor([n], dtype=torch.int32, device="cuda"))
    assert torch.equal(a.cache.pages, b.cache.pages)
    assert torch.equal(a.cache.bounds.view(torch.int16), b.cache.bounds.view(torch.int16))


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("G", [32, 64])
def test_awkward_values(dtype, G):
    """Constant groups, zeros, the type's extremes, subnormals; infinities and NaN poison their
    own group only."""
    w = World(64, G, 16, dtype, 1, [16])
    k, big, tiny = w.k[0], torch.finfo(dtype).max, torch.finfo(dtype).smallest_normal
    k[0] = 0.0
    k[1] = 3.25
    k[2, 0, :32], k[2, 0, 32:] = big, -big
    k[3, 0, ::2], k[3, 0, 1::2] = big, -big
    k[4] = k[4] * tiny
    k[5, 0, 3] = math.inf
    k[6, 0, 40] = math.nan
    k[7, 0, 0], k[7, 0, 1] = -math.inf, math.inf
    k[8] = -0.0
    k[9] = big
    w.v[0] = k.flip(0).contiguous()
    w.fill()
    ko, vo = torch.empty_like(k)[None], torch.empty_like(k)[None]
    w.cache.read(ko, vo, **w.batch)
    kx, vx = w.values(0)
    # 8 s and the sums are fp32 in the kernel and 64-bit here: the same after rounding, as s (u - 8) is exact
    assert same_bits(ko[0], kx.float().to(dtype)) and same_bits(vo[0], vx.float().to(dtype))
    assert torch.isnan(ko[0, 5, 0, :32]).all() and (G == 64 or torch.isfinite(ko[0, 5, 0, 32:]).all())


def test_strides_rows_that_are_no_tokens_and_bad_tables():
    w = World(128, 64, 16, BF, 2, [40, 5, 0])
    n = 48  # more rows than tokens: the first ones are before the sequence
    packed = torch.randn(3, n, 3, 2, 128, device="cuda").to(BF)  # [.., (q, k, v), heads, D]
    k, v = packed[:, :, 1], packed[:, :, 2]
    guard = w.cache.pages.clone()
    w.cache.append(k, v, **w.batch)
    out = torch.full((3, 2, n, 2, 128), 7.0, dtype=BF, device="cuda")
    w.cache.read(out[:, 0], out[:, 1], **w.batch)
    for i, length in enumerate(w.lens):
        for x, o in ((k, out[:, 0]), (v, out[:, 1])):
            assert (o[i, :n - length] == 0).all()
            assert same_bits(o[i, n - length:], ref.values(x[i, n - length:], 64).to(BF))
    # table entries outside the pool and lengths beyond the table: nothing is written, zeros are read
    table = w.table.clone()
    table[0, 1], table[0, 2], table[1, 0] = -5, w.cache.pages.shape[1], 1 << 30
    used = w.table[0, 0].item()
    w.cache.pages.copy_(guard)
    lens = torch.tensor([40, 5, 1000], dtype=torch.int32, device="cuda")
    w.cache.append(k, v, table=table, lens=lens)
    changed = (w.cache.pages != guard).flatten(2).any(-1).any(0).nonzero().flatten().tolist()
    assert changed == [used]
    w.cache.read(out[:, 0], out[:, 1], table=table, lens=lens)
    assert (out[0, :, 24:] == 0).all() and (out[1] == 0).all() and (out[2] == 0).all()


def test_offsets_past_32_bits():
    from moe_expert_layer_sorted_gb300 import KVCache
    cache = KVCache.allocate(70000, kv_heads=8, head_dim=128, page_size=64, dtype=BF)
    assert cache.pages.numel() > 1 << 32
    lens = torch.tensor([130], dtype=torch.int32, device="cuda")
    table = torch.tensor([[69999, 3, 65001]], dtype=torch.int32, device="cuda")
    k, v, q = (torch.randn(1, 130, 8, 128, device="cuda").to(BF) for _ in range(3))
    cache.append(k, v, table=table, lens=lens)
    ko, vo, out = torch.empty_like(k), torch.empty_like(k), torch.empty_like(k)
    cache.read(ko, vo, table=table, lens=lens)
    kx, vx = ref.values(k[0], 64), ref.values(v[0], 64)
    assert same_bits(ko[0], kx.to(BF)) and same_bits(vo[0], vx.to(BF))
    seen = torch.ones(130, 130, device="cuda").tril().bool()
    for rows in (1, 130):
        o = torch.empty_like(q[:, -rows:])
        cache.attention(q[:, -rows:], o, table=table, lens=lens)
        want, _, tol, _ = ref.attention(q[0, -rows:], kx, vx, seen[-rows:], 1 / math.sqrt(128))
        check(o[0], want, tol)


# ----------------------------------------------------------------------------- attention

def run_attention(w, counts, q_heads, causal=True, ragged=True, scale=None, lse=True):
    N = sum(counts)
    q = w.rand(N, q_heads, w.D)
    out, ls = torch.full_like(q, 9.0), torch.full((N, q_heads), 9.0, device="cuda")
    batch = dict(w.batch)
    if ragged:
        batch.update(starts=starts_of(counts), max_new=max(counts))
        w.cache.attention(q, out, causal=causal, scale=scale, lse=ls if lse else None, **batch)
    else:
        shape = (len(counts), counts[0], q_heads, w.D)
        w.cache.attention(q.view(shape), out.view(shape), causal=causal, scale=scale, lse=ls if lse else None, **batch)
    at, sc = 0, scale if scale is not None else 1 / math.sqrt(w.D)
    for i, n in enumerate(counts):
        L = w.lens[i]
        pos = torch.arange(L - n, L, device="cuda")[:, None]
        seen = (torch.arange(L, device="cuda")[None] <= pos) if causal else torch.ones(n, L, dtype=torch.bool, device="cuda")
        want, wl, tol, ltol = ref.attention(q[at:at + n], *w.values(i), seen, sc)
        check(out[at:at + n], want, tol, f"sequence {i}")
        if lse:
            empty = torch.isinf(wl)
            assert (ls[at:at + n][empty] == -math.inf).all()
            assert ((ls[at:at + n].double() - wl)[~empty].abs() <= ltol[~empty] + 1e-5).all()
        at += n


@pytest.mark.parametrize("D,G,P,dtype", GEOMETRY)
@pytest.mark.parametrize("per", [1, 3, 8])
def test_attention_of_single_tokens(D, G, P, dtype, per):
    lens = [1, 2, 15, 16, 17, 63, 64, 65, 127, 128, 129, 257, 0, 1000, 31]
    run_attention(World(D, G, P, dtype, 2, lens, seed=per).fill(), [1] * len(lens), 2 * per, ragged=False)


@pytest.mark.parametrize("per", [2, 7, 16, 24])
@pytest.mark.parametrize("n", [2, 3, 5])
def test_attention_of_a_few_tokens(per, n):
    """Rows before a sequence's first token see nothing: zeros, lse -inf."""
    w = World(128, 64, 16, BF, 1, [1, 3, n, 50, 300], seed=n).fill()
    run_attention(w, [n] * 5, per, ragged=False)
    run_attention(w, [1, n, 1, n, 2], per)


@pytest.mark.parametrize("D,G,P,dtype", GEOMETRY)
@pytest.mark.parametrize("per,counts,extra", [(1, [130, 1, 64], [0, 5, 300]), (4, [33, 200], [100, 0]), (8, [17], [7]),
                                              (3, [129, 40], [0, 1000])])
def test_attention_of_prompts(D, G, P, dtype, per, counts, extra):
    w = World(D, G, P, dtype, 2, [a + b for a, b in zip(counts, extra)], seed=per).fill()
    run_attention(w, counts, 2 * per)


@pytest.mark.parametrize("counts,lens", [([40, 300], [10, 280]), ([100, 0, 64], [0, 30, 64])])
def test_attention_rows_before_the_sequence_and_sequences_without_rows(counts, lens):
    run_attention(World(128, 64, 32, BF, 2, lens, seed=4).fill(), counts, 8)
    run_attention(World(64, 32, 32, FP, 2, lens, seed=4).fill(), counts, 2)


@pytest.mark.parametrize("counts", [[1, 1], [3, 3], [150, 70]])
def test_attention_without_causal_mask(counts):
    run_attention(World(128, 64, 64, BF, 2, [333, 190], seed=9).fill(), counts, 8, causal=False)


@pytest.mark.parametrize("counts", [[1], [4], [96]])
def test_large_scores(counts):
    """Scores of several hundred: the running maximum carries the softmax."""
    w = World(128, 64, 64, BF, 1, [700], seed=3).fill()
    run_attention(w, counts, 4, scale=3.0)
    run_attention(w, counts, 4, scale=-0.5)
    run_attention(w, counts, 4, scale=0.0)


@pytest.mark.parametrize("dtype,big,small", [(BF, 1e9, 1e-9), (FP, 6e4, 1e-4)])
@pytest.mark.parametrize("n", [1, 3, 80])
def test_keys_and_queries_of_any_size(dtype, big, small, n):
    """Tiny and huge keys beside ordinary ones, values up to the type's largest, tiny and huge
    queries: scores of ordinary size throughout."""
    w = World(128, 64, 32, dtype, 2, [300, 300, 300], seed=n)
    w.k[0][5:200:7] *= small
    w.k[0][9] = 0.0
    w.k[1] = (w.k[1].float().clamp(-1, 1) * big).to(dtype)
    w.k[2] = (w.k[2].float() * small).to(dtype)
    w.v[2][::3] = (w.v[2][::3].float().clamp(-1, 1) * torch.finfo(dtype).max).to(dtype)
    w.v[2][::3, :, ::2] = -torch.finfo(dtype).max
    w.fill()
    q = w.rand(3, n, 8, 128)
    q[1] = (q[1].float() / big).to(dtype)
    q[2] = (q[2].float() / small).to(dtype)
    out = torch.empty_like(q)
    w.cache.attention(q, out, **w.batch)
    for i in range(3):
        seen = torch.arange(300, device="cuda")[None] <= torch.arange(300 - n, 300, device="cuda")[:, None]
        want, _, tol, _ = ref.attention(q[i], *w.values(i), seen, 1 / math.sqrt(128))
        check(out[i], want, tol, f"sequence {i}")


def test_long_sequences_are_split_and_joined():
    run_attention(World(128, 64, 64, BF, 2, [20011], seed=5).fill(), [1], 16, ragged=False)
    run_attention(World(64, 32, 16, FP, 1, [9000, 40], seed=6).fill(), [1, 1], 4, ragged=False)
    run_attention(World(128, 128, 128, FP, 1, [20011, 3], seed=7).fill(), [2, 3], 2)


@pytest.mark.parametrize("D,G,P,dtype,per", [(128, 64, 64, BF, 4), (64, 32, 16, FP, 1), (128, 128, 128, FP, 8)])
def test_prompts_over_long_contexts(D, G, P, dtype, per):
    """Few rows and many tokens: the tokens are cut into stretches, some rows see none of the last."""
    run_attention(World(D, G, P, dtype, 1, [9001, 700, 20], seed=per).fill(), [50, 300, 40], per)
    w = World(D, G, P, dtype, 2, [4003], seed=per + 1)
    w.v[0][17, 1, 5] = math.inf
    w.fill()
    q = w.rand(1, 60, 2 * per, D)
    out = torch.empty_like(q)
    w.cache.attention(q, out, **w.batch)
    assert torch.isnan(out[0, :, per:, :G]).all() and torch.isfinite(out[0, :, :per]).all()
    assert torch.isfinite(out[0, :, per:, G:]).all()


def test_many_short_sequences():
    rng = np.random.default_rng(0)
    lens = rng.integers(0, 90, 300).tolist()
    run_attention(World(128, 64, 16, BF, 2, lens, seed=8).fill(), [1] * 300, 8, ragged=False)


@pytest.mark.parametrize("n", [1, 2, 90])
def test_poisoned_and_missing_tokens(n):
    """A NaN value reaches the rows that see it and no other; tokens on missing pages are as
    if masked."""
    w = World(128, 64, 16, BF, 2, [100, 100], seed=11)
    w.v[0][99, 1, 70] = math.nan
    w.fill()
    q, out = w.rand(2, n, 4, 128), torch.empty(2, n, 4, 128, dtype=BF, device="cuda")
    w.cache.attention(q, out, **w.batch)
    assert torch.isnan(out[0, -1, 2:, 64:]).all()
    assert torch.isfinite(out[0, -1, :2]).all() and torch.isfinite(out[0, :-1]).all() and torch.isfinite(out[1]).all()
    table = w.table.clone()
    table[1, 2], table[1, 6] = -1, 1 << 29
    table[0] = -1
    lse = torch.empty(2 * n, 4, device="cuda")
    w.cache.attention(q, out, table=table, lens=w.lens_t, lse=lse)
    seen = torch.arange(100, device="cuda")[None] <= torch.arange(100 - n, 100, device="cuda")[:, None]
    seen[:, 32:48] = False
    seen[:, 96:] = False
    want, _, tol, _ = ref.attention(q[1], *w.values(1), seen, 1 / math.sqrt(128))
    check(out[1], want, tol)
    assert (out[0] == 0).all() and (lse[:n] == -math.inf).all()
    # lengths beyond the table's pages: what the table holds
    w.cache.attention(q, out, table=w.table[:, :2], lens=w.lens_t)
    want, _, tol, _ = ref.attention(q[1], *(x[:32] for x in w.values(1)),
                                    seen[:, :32] | (torch.arange(100 - n, 100, device="cuda")[:, None] >= 32), 1 / math.sqrt(128))
    check(out[1], want, tol)


@pytest.mark.parametrize("n", [1, 70])
def test_strided_queries_and_outputs(n):
    w = World(128, 64, 32, BF, 2, [150, 90], seed=12).fill()
    big = torch.randn(2, n, 8 + 2 + 2, 128, device="cuda").to(BF)
    q = big[:, :, :8]
    out = torch.full((2, 8, n, 128), 3.0, dtype=BF, device="cuda").transpose(1, 2)  # [2, n, 8, 128], heads outermost
    w.cache.attention(q, out, **w.batch)
    plain = torch.empty(2, n, 8, 128, dtype=BF, device="cuda")
    w.cache.attention(q.contiguous(), plain, **w.batch)
    assert torch.equal(out, plain)


def test_layers_are_apart():
    w = World(128, 64, 16, BF, 2, [50], layers=3, layer=2).fill()
    assert (w.cache.pages[:2] == 0xFF).all()
    run_attention(w, [1], 4, ragged=False)


def test_repeatable_streams_and_graph():
    w = World(128, 64, 64, BF, 4, [3001, 77, 512], seed=13).fill()
    q = w.rand(3, 1, 16, 128)
    outs = [torch.empty_like(q) for _ in range(6)]
    w.cache.attention(q, outs[0], **w.batch)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for i in range(1, 5):  # the workspace is shared: calls on different streams follow one another
        w.cache.attention(q, outs[i], stream=side if i % 2 else None, **w.batch)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        w.cache.attention(q, outs[5], **w.batch)
    q2 = q.clone()
    for _ in range(3):
        outs[5].zero_()
        g.replay()
    torch.cuda.synchronize()
    for o in outs[1:]:
        assert torch.equal(outs[0], o)
    assert torch.equal(q, q2)


# ----------------------------------------------------------------------------- selection

@pytest.mark.parametrize("D,G,P,dtype", [(64, 32, 16, FP), (128, 64, 32, BF)])
@pytest.mark.parametrize("budget,first,last", [(1, 0, 1), (5, 1, 1), (12, 2, 3), (200, 1, 1)])
def test_selection(D, G, P, dtype, budget, first, last):
    lens = [1, P, 11 * P + 3, 150 * P - 1, 0]
    w = World(D, G, P, dtype, 2, lens, seed=budget).fill()
    for n, per in ((1, 1), (3, 4)):
        q = w.rand(len(lens), n, 2 * per, D)
        pages = torch.full((len(lens) * n, 2, budget), 99, dtype=torch.int32, device="cuda")
        w.cache.select(q, pages, keep_first=first, keep_last=last, **w.batch)
        got = pages.view(len(lens), n, 2, budget).tolist()
        for i, L in enumerate(lens):
            ends = w.cache.bounds[0][w.table[i].long().clamp_min(0)].cpu()
            for j in range(n):
                pos = L - n + j
                for h in range(2):
                    want = ref.select(q[i, j, h * per:(h + 1) * per].cpu(), ends[:, h, 0], ends[:, h, 1],
                                      pos // P + 1 if pos >= 0 else 0, budget, first, last)
                    assert got[i][j][h] == want
        # attention over the choice
        out = torch.empty_like(q)
        w.cache.attention(q, out, pages=pages, **w.batch)
        for i, L in enumerate(lens):
            seen = torch.zeros(n, 2, L, dtype=torch.bool, device="cuda")
            for j in range(n):
                for h in range(2):
                    at = torch.arange(L, device="cuda")
                    chosen = torch.tensor(got[i][j][h], device="cuda")
                    seen[j, h] = torch.isin(at // P, chosen) & (at <= L - n + j)
            want, _, tol, _ = ref.attention(q[i], *w.values(i), seen, 1 / math.sqrt(D))
            check(out[i], want, tol)


def test_selection_ties_nan_and_many_pages():
    w = World(64, 32, 16, BF, 1, [16 * 700], seed=1)
    g = torch.Generator().manual_seed(5)
    hi = torch.randint(-2, 3, (700, 64), generator=g).to(BF)  # few distinct scores: many ties
    hi[::3] = hi[0]
    lo = hi - 1
    hi[50, 3], hi[51, 4], lo[52, 5], hi[53] = math.nan, math.inf, -math.inf, -0.0
    w.cache.bounds[0, w.table[0].long(), 0, 0], w.cache.bounds[0, w.table[0].long(), 0, 1] = hi.cuda(), lo.cuda()
    for budget in (3, 64, 233, 234, 698, 699):
        q = w.rand(1, 1, 2, 64).round()
        pages = torch.empty(1, 1, budget, dtype=torch.int32, device="cuda")
        w.cache.select(q, pages, **w.batch)
        assert pages[0, 0].tolist() == ref.select(q[0, 0].cpu(), hi, lo, 700, budget, 1, 1)


def test_selection_of_ragged_rows_in_chunks():
    """More rows than the workspace holds scores for at once."""
    w = World(64, 64, 16, FP, 8, [900, 2100], seed=2).fill()
    table = torch.full((2, 3000), -1, dtype=torch.int32, device="cuda")
    table[:, :w.cols] = w.table
    counts = [300, 200]
    q = w.rand(500, 8, 64)
    pages = torch.empty(500, 8, 6, dtype=torch.int32, device="cuda")
    w.cache.select(q, pages, table=table, lens=w.lens_t, starts=starts_of(counts), max_new=300)
    got = pages.cpu().tolist()
    for r in (0, 1, 150, 299, 300, 301, 444, 499):
        i, j = (0, r) if r < 300 else (1, r - 300)
        pos = w.lens[i] - counts[i] + j
        ends = w.cache.bounds[0][w.table[i].long().clamp_min(0)].cpu()
        for h in (0, 3, 7):
            assert got[r][h] == ref.select(q[r, h:h + 1].cpu(), ends[:, h, 0], ends[:, h, 1], pos // 16 + 1, 6, 1, 1)


def test_choice_with_foreign_and_future_pages():
    """Entries outside the sequence, beyond the row and negative ones are skipped."""
    w = World(128, 64, 16, BF, 1, [60], seed=3).fill()
    q, out = w.rand(1, 2, 2, 128), torch.empty(1, 2, 2, 128, dtype=BF, device="cuda")
    pages = torch.tensor([[[2, -1, 40, 3, 1 << 28]], [[-1, -7, 9, 77, 1 << 30]]], dtype=torch.int32, device="cuda")
    w.cache.attention(q, out, pages=pages, **w.batch)
    seen = torch.zeros(1, 60, dtype=torch.bool, device="cuda")
    seen[0, 32:59] = True
    want, _, tol, _ = ref.attention(q[0, :1], *w.values(0), seen, 1 / math.sqrt(128))
    check(out[0, :1], want, tol)
    assert (out[0, 1] == 0).all()


# ------------------------------------------------------------------------------ refusals

def test_refusals():
    from moe_expert_layer_sorted_gb300 import KVCache, MoeError
    w = World(128, 64, 16, BF, 2, [20], seed=1).fill()
    c, b = w.cache, w.batch
    q, kv = w.rand(1, 1, 4, 128), w.rand(1, 1, 2, 128)
    o = torch.empty_like(q)
    pages = torch.zeros(1, 2, 4, dtype=torch.int32, device="cuda")
    odd = torch.zeros(4 * 128 + 8, dtype=BF, device="cuda")[1:513].view(1, 1, 4, 128)
    bad = [
        lambda: c.append(kv[..., :64], kv, **b), lambda: c.append(kv, kv.half(), **b), lambda: c.append(q, q, **b),
        lambda: c.append(kv.cpu(), kv.cpu(), **b), lambda: c.append(kv, kv[:, :, :1], **b),
        lambda: c.read(kv, kv.expand(1, 1, 2, 128)[:, :, :1].expand(1, 1, 2, 128), **b),
        lambda: c.attention(q, o, table=w.table.long(), lens=w.lens_t),
        lambda: c.attention(q, o, table=w.table, lens=w.lens_t.cpu()),
        lambda: c.attention(q, o, table=w.table, lens=torch.zeros(2, dtype=torch.int32, device="cuda")),
        lambda: c.attention(q[:, :, :3], o[:, :, :3], **b),              # 3 heads over 2
        lambda: c.attention(q, q, **b), lambda: c.attention(odd, o, **b), lambda: c.attention(q, odd, **b),
        lambda: c.attention(q, o, scale=math.nan, **b), lambda: c.attention(q, o, scale=math.inf, **b),
        lambda: c.attention(q, o, table=w.table, lens=w.lens_t, layer=1),
        lambda: c.attention(q, o, lse=torch.empty(3, device="cuda"), **b),
        lambda: c.attention(q, o, pages=pages.long(), **b), lambda: c.attention(q, o, pages=pages[:, :1].contiguous(), **b),
        lambda: c.attention(q[0], o[0], **b),                            # ragged tensor without starts
        lambda: c.attention(q, o, max_new=1 + 1, **b),
        lambda: c.attention(q[0], o[0], starts=torch.zeros(3, dtype=torch.int32, device="cuda"), **b),
        lambda: c.select(q, pages, keep_first=3, keep_last=2, **b), lambda: c.select(q, pages, keep_last=0, **b),
        lambda: c.select(q, pages, table=torch.zeros(1, 3 << 20, dtype=torch.int32, device="cuda"), lens=w.lens_t),
        lambda: KVCache.allocate(4, kv_heads=2, head_dim=96), lambda: KVCache.allocate(4, kv_heads=2, head_dim=64, group_size=128),
        lambda: KVCache.allocate(4, kv_heads=2, head_dim=64, page_size=48),
        lambda: KVCache.allocate(4, kv_heads=2, head_dim=64, dtype=torch.float32),
        lambda: KVCache(c.pages[..., :16], page_size=16, head_dim=128),
        lambda: KVCache(c.pages, page_size=16, head_dim=128, bounds=c.bounds.half()),
        lambda: KVCache(c.pages, page_size=32, head_dim=128),
    ]
    for i, f in enumerate(bad):
        with pytest.raises(MoeError):
            f()
            pytest.fail(f"case {i} was not refused")
    plain = KVCache(c.pages, page_size=16, head_dim=128)  # without bounds
    with pytest.raises(MoeError, match="bounds"):
        plain.select(q, pages, **b)
    # no rows, no sequences: nothing to do
    c.attention(q[:, :0], o[:, :0], **b)
    c.append(kv[:0], kv[:0], table=w.table[:0], lens=w.lens_t[:0])
    torch.cuda.synchronize()


def test_calls_of_the_binding():
    from moe_expert_layer_sorted_gb300 import MoeError
    w = World(64, 32, 16, FP, 2, [40], seed=3).fill()
    q = w.rand(1, 1, 4, 64)
    out = [torch.empty_like(q) for _ in range(4)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for o, stream in zip(out, (None, torch.cuda.current_stream().cuda_stream, side, side.cuda_stream)):
        w.cache.attention(q, o, stream=stream, **w.batch)  # the current one, an address, a stream
    with torch.cuda.stream(side):
        again = torch.empty_like(q)
        w.cache.attention(q, again, **w.batch)
    torch.cuda.synchronize()
    assert all(torch.equal(out[0], o) for o in out[1:] + [again])
    for bad in (dict(stream="0"), dict(layer="0"), dict(scale="1"), dict(layer=1 << 40)):
        with pytest.raises((MoeError, TypeError, AttributeError, OverflowError)):
            w.cache.attention(q, out[0], **{**w.batch, **bad})
    for q_, o_ in ((None, out[0]), (q, None), (q.cpu().numpy(), out[0]), (q[0, 0], out[0]), (q, out[0].expand(2, 1, 4, 64))):
        with pytest.raises(MoeError):
            w.cache.attention(q_, o_, **w.batch)
    with pytest.raises(MoeError):  # a destination whose rows are one row
        w.cache.read(*(torch.empty(1, 1, 1, 64, dtype=FP, device="cuda").expand(1, 1, 2, 64) for _ in "kv"), **w.batch)
    w.cache.close()
    w.cache.close()
    with pytest.raises(MoeError, match="closed"):
        w.cache.attention(q, out[0], **w.batch)


def test_short_rows_are_chosen_on_two_streams_at_once():
    w = World(128, 64, 16, BF, 2, [900, 333], seed=9).fill()
    q = w.rand(2, 1, 8, 128)
    chosen = [torch.full((2, 2, 7), -9, dtype=torch.int32, device="cuda") for _ in range(8)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    for i, pages in enumerate(chosen):
        w.cache.select(q, pages, stream=streams[i % 2], **w.batch)
    torch.cuda.synchronize()
    assert (chosen[0] >= 0).all() and all(torch.equal(chosen[0], c) for c in chosen[1:])
