"""The 8-bit key/value cache on the GPU: what it stores, attention, the weight of tokens and eviction, against
the plain implementation, over head layouts, lengths, masks and strides where they can go wrong."""
import math

import numpy as np
import pytest
import torch

import kv8_reference as ref

pytestmark = pytest.mark.gpu

BF, FP = torch.bfloat16, torch.float16
GEOMETRY = [(64, 16, BF), (64, 64, FP), (128, 32, FP), (128, 64, BF), (128, 256, BF), (128, 128, FP)]


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def starts_of(counts):
    return ints(np.concatenate([[0], np.cumsum(counts)]).tolist())


def same_bits(a, b):
    """Equal values, NaN where NaN."""
    return torch.equal(torch.isnan(a), torch.isnan(b)) and torch.equal(a.nan_to_num(7.0), b.nan_to_num(7.0))


class World:
    """Sequences with known keys and values in a cache whose free memory is NaN."""

    def __init__(self, D, P, dtype, heads, lens, seed=0, spare=3, layers=1, layer=0):
        from moe_expert_layer_sorted_gb300 import KVCache8
        self.D, self.P, self.dtype, self.heads, self.lens, self.layer = D, P, dtype, heads, list(lens), layer
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.g = g
        need = [-(-n // P) for n in lens]
        self.cols = max(need + [1])
        total = sum(need) + spare
        self.cache = KVCache8.allocate(total, kv_heads=heads, head_dim=D, page_size=P, dtype=dtype, layers=layers)
        self.cache.pages.fill_(0xFF)  # steps of all ones: NaN
        self.cache.mass.fill_(math.nan)
        ids = torch.randperm(total, generator=g, device="cuda").int()
        self.table = torch.full((len(lens), self.cols), -1, dtype=torch.int32, device="cuda")
        at = 0
        for i, n in enumerate(need):
            self.table[i, :n] = ids[at:at + n]
            at += n
        self.lens_t = ints(self.lens)
        scale = torch.exp(0.5 * torch.randn(heads, D, generator=g, device="cuda"))
        self.k = [(torch.randn(n, heads, D, generator=g, device="cuda") * scale).to(dtype) for n in lens]
        self.v = [self.rand(n, heads, D) for n in lens]
        self.stored = [ref.Stored(heads, D) for _ in lens]

    def rand(self, *shape):
        return torch.randn(*shape, generator=self.g, device="cuda").to(self.dtype)

    def fill(self, pieces=None):
        """Each sequence in one call, or in calls of the given sizes, the last again and again."""
        for i, n in enumerate(self.lens):
            at, todo = 0, list(pieces or [n])
            while at < n:
                m = min(n - at, todo[0])
                todo = todo[1:] or todo
                self.cache.append(self.k[i][None, at:at + m], self.v[i][None, at:at + m], table=self.table[i:i + 1],
                                  layer=self.layer, lens=ints([at + m]))
                self.stored[i].append(self.k[i][at:at + m], self.v[i][at:at + m])
                at += m
        return self

    @property
    def batch(self):
        return dict(table=self.table, lens=self.lens_t, layer=self.layer)

    def read(self, lens=None):
        lens = self.lens if lens is None else lens
        k, v = (torch.full((sum(lens), self.heads, self.D), 5.0, dtype=self.dtype, device="cuda") for _ in range(2))
        self.cache.read(k, v, table=self.table, layer=self.layer, lens=ints(lens), starts=starts_of(lens), max_new=max(lens + [1]))
        return k.split(lens), v.split(lens)

    def holds(self, lens=None):
        """What is read is what is stored."""
        for st, k, v in zip(self.stored, *self.read(lens)):
            kx, vx = st.values()
            assert same_bits(k, kx.float().to(self.dtype)) and same_bits(v, vx.float().to(self.dtype))

    def mass_of(self, i, n=None):
        """[tokens, H]"""
        n = self.lens[i] if n is None else n
        j = torch.arange(n, device="cuda")
        return self.cache.mass[self.layer][self.table[i].long()[j // self.P], :, j % self.P]

    def set_mass(self, i, mass):
        j = torch.arange(len(mass), device="cuda")
        self.cache.mass[self.layer][self.table[i].long()[j // self.P], :, j % self.P] = mass


# ------------------------------------------------------------------------ write and read

@pytest.mark.parametrize("D,P,dtype", GEOMETRY)
def test_layout_and_codes(D, P, dtype):
    w = World(D, P, dtype, 2, [P + 19]).fill()
    st = w.stored[0]
    for pos0 in range(0, P + 19, 16):
        page, blk = int(w.table[0, pos0 // P]), pos0 % P // 16
        for h in range(2):
            u, s, marks = ref.block_bytes(w.cache.pages[0, page, h, blk].cpu().numpy(), D)
            n = min(16, P + 19 - pos0)
            assert np.array_equal(u[:, :n], st.u[:, pos0:pos0 + n, h].cpu().numpy())
            assert np.array_equal(s.astype(np.float64), st.s[:, pos0 // 16, h].cpu().numpy()) and not marks.any()


@pytest.mark.parametrize("D,P,dtype", GEOMETRY)
@pytest.mark.parametrize("pieces", [[1], [5, 1, 3, 2], [37, 1], [16, 7]])
def test_append_in_pieces_then_read(D, P, dtype, pieces):
    """Older tokens of a block are turned where its step grows."""
    w = World(D, P, dtype, 3, [P + 23, 3, 70]).fill(pieces)
    w.holds()
    for i in range(3):
        assert (w.mass_of(i) == 0).all()
    assert torch.isnan(w.cache.mass).sum() == (w.cache.mass.numel() - 3 * sum(w.lens))


def test_ragged_and_uniform_writes():
    w = World(128, 32, BF, 2, [50, 33, 41, 17])
    n = [18, 1, 0, 16]
    for i, m in enumerate(n):
        w.cache.append(w.k[i][None, :w.lens[i] - m], w.v[i][None, :w.lens[i] - m], table=w.table[i:i + 1], lens=ints([w.lens[i] - m]))
        w.stored[i].append(w.k[i][:w.lens[i] - m], w.v[i][:w.lens[i] - m])
        if m:
            w.stored[i].append(w.k[i][-m:], w.v[i][-m:])
    k, v = (torch.cat([x[i][len(x[i]) - m:] for i, m in enumerate(n)]) for x in (w.k, w.v))
    w.cache.append(k, v, starts=starts_of(n), max_new=18, **w.batch)
    w.holds()


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("pieces", [None, [1], [7, 2]])
def test_awkward_values(dtype, pieces):
    """Zeros, the type's extremes, subnormals, halves of the largest (ties); infinities and NaN mark their own
    token and head only."""
    n = 16 * 8
    w = World(64, 16, dtype, 2, [n])
    k, big, info = w.k[0], torch.finfo(dtype).max, torch.finfo(dtype)
    b = k.view(8, 16, 2, 64)
    b[0] = 0.0
    b[1, :, :, ::2], b[1, :, :, 1::2] = big, -big
    b[2] *= info.smallest_normal
    b[3] = b[3].sign() * info.smallest_normal * info.eps  # the smallest subnormal
    b[4, 3, 0, 3], b[4, 5, 1, 40], b[4, 6, 0, 0], b[4, 6, 0, 1] = math.inf, math.nan, -math.inf, math.inf
    b[5, :, 0] = torch.arange(64, device="cuda").to(dtype) - 32  # of 32: 63.5 and -63.5 are ties
    b[5, :, 1] = 127.0
    b[5, 4:, 1, :] = torch.arange(64, device="cuda").to(dtype) * 0.5
    b[6, :8] = -0.0
    b[7] *= 1e-3
    b[7, 15] = big
    w.v[0] = k.view(8, 16, 2, 64).flip(0).reshape(n, 2, 64).contiguous()
    w.fill(pieces)
    w.holds()
    (ko,), _ = w.read()
    bad = torch.isnan(ko).view(8, 16, 2, 64)
    assert bad[4, 3, 0].all() and bad[4, 5, 1].all() and bad[4, 6, 0].all() and int(bad.sum()) == 3 * 64


def test_every_16_bit_value_beside_a_larger_one():
    """Codes of all finite bf16 values below steps of many sizes: quotients near halves among them."""
    every = torch.arange(0, 0x7f80, device="cuda", dtype=torch.int32).to(torch.int16).view(BF)
    n = 32640 // 64  # of 64 channels
    for shift in (0, 1, 7, 40):
        x = every.view(n, 1, 64).clone()
        x[::16, 0, :1] = every.view(n, 64)[min(shift, n - 1) * 1 if shift else n - 1, 63]
        w = World(64, 64, BF, 1, [n], seed=shift)
        w.k[0], w.v[0] = x, -x.flip(0).contiguous()
        w.fill()
        w.holds()


def test_strides_rows_that_are_no_tokens_and_bad_tables():
    w = World(128, 16, BF, 2, [40, 5, 0])
    n = 48  # more rows than tokens: the first ones are before the sequence
    packed = torch.randn(3, n, 3, 2, 128, device="cuda").to(BF)  # [.., (q, k, v), heads, D]
    k, v = packed[:, :, 1], packed[:, :, 2]
    guard, mass = w.cache.pages.clone(), w.cache.mass.clone()
    w.cache.append(k, v, **w.batch)
    out = torch.full((3, 2, n, 2, 128), 7.0, dtype=BF, device="cuda")
    w.cache.read(out[:, 0], out[:, 1], **w.batch)
    for i, length in enumerate(w.lens):
        st = ref.Stored(2, 128).append(k[i, n - length:], v[i, n - length:]) if length else ref.Stored(2, 128)
        for x, o in zip(st.values(), (out[:, 0], out[:, 1])):
            assert (o[i, :n - length] == 0).all()
            assert same_bits(o[i, n - length:], x.float().to(BF))
    # table entries outside the pool and lengths beyond the table: nothing is written, zeros are read
    table = w.table.clone()
    table[0, 1], table[0, 2], table[1, 0] = -5, w.cache.pages.shape[1], 1 << 30
    used = w.table[0, 0].item()
    w.cache.pages.copy_(guard)
    w.cache.mass.copy_(mass)
    lens = ints([40, 5, 1000])
    w.cache.append(k, v, table=table, lens=lens)
    changed = (w.cache.pages != guard).flatten(2).any(-1).any(0).nonzero().flatten().tolist()
    assert changed == [used]
    assert (~torch.isnan(w.cache.mass)).flatten(2).any(-1).any(0).nonzero().flatten().tolist() == [used]
    w.cache.read(out[:, 0], out[:, 1], table=table, lens=lens)
    assert (out[0, :, 24:] == 0).all() and (out[1] == 0).all() and (out[2] == 0).all()


# ----------------------------------------------------------------------------- attention

def causal(n, L):
    return torch.arange(L, device="cuda")[None] <= torch.arange(L - n, L, device="cuda")[:, None]


def expected(w, i, q, scale=None, is_causal=True):
    n, L = len(q), w.stored[i].length
    k, v = w.stored[i].values()
    real = torch.arange(L - n, L, device="cuda")[:, None] >= 0  # rows before the first token see nothing
    seen = causal(n, L) if is_causal else real.expand(n, L)
    return ref.attention(q, k, v, w.stored[i].steps()[1], seen, scale if scale is not None else 1 / math.sqrt(w.D))


def run_attention(w, counts, q_heads, is_causal=True, ragged=True, scale=None, lse=True, weigh=False, q=None):
    N = sum(counts)
    q = w.rand(N, q_heads, w.D) if q is None else q
    out, ls = torch.full_like(q, 9.0), torch.full((N, q_heads), 9.0, device="cuda")
    batch = dict(w.batch, causal=is_causal, scale=scale, lse=ls if lse else None, weigh=weigh)
    before = [w.mass_of(i).double() for i in range(len(counts))]
    if ragged:
        w.cache.attention(q, out, starts=starts_of(counts), max_new=max(counts), **batch)
    else:
        shape = (len(counts), counts[0], q_heads, w.D)
        w.cache.attention(q.view(shape), out.view(shape), **batch)
    for i, (x, o, l) in enumerate(zip(q.split(counts), out.split(counts), ls.split(counts))):
        want = expected(w, i, x, scale, is_causal)
        ref.check(o, l if lse else None, want, f"sequence {i}")
        if weigh:
            add, tol = ref.masses(want, w.heads)
            now = w.mass_of(i).double()
            off = (now - before[i] - add).abs() - (tol + 2.0 ** -23 * now.abs())
            assert (off <= 0).all(), f"mass of sequence {i}: {float(off.max())} beyond its bound"
    return out, ls


@pytest.mark.parametrize("D,P,dtype", GEOMETRY)
@pytest.mark.parametrize("per", [1, 3, 8])
def test_attention_of_single_tokens(D, P, dtype, per):
    lens = [1, 2, 15, 16, 17, 63, 64, 65, 127, 128, 129, 257, 0, 1000, 31]
    run_attention(World(D, P, dtype, 2, lens, seed=per).fill(), [1] * len(lens), 2 * per, ragged=False)


@pytest.mark.parametrize("per", [2, 7, 16, 24])
@pytest.mark.parametrize("n", [2, 3, 5])
def test_attention_of_a_few_tokens(per, n):
    """Rows before a sequence's first token see nothing: zeros, lse -inf."""
    w = World(128, 16, BF, 1, [1, 3, n, 50, 300], seed=n).fill()
    run_attention(w, [n] * 5, per, ragged=False)
    run_attention(w, [1, n, 1, n, 2], per)


@pytest.mark.parametrize("D,P,dtype", GEOMETRY)
@pytest.mark.parametrize("per,counts,extra", [(1, [130, 1, 64], [0, 5, 300]), (4, [33, 200], [100, 0]), (8, [17], [7]),
                                              (3, [129, 40], [0, 1000])])
def test_attention_of_prompts(D, P, dtype, per, counts, extra):
    w = World(D, P, dtype, 2, [a + b for a, b in zip(counts, extra)], seed=per).fill()
    run_attention(w, counts, 2 * per)


@pytest.mark.parametrize("n", [1, 40])
def test_attention_without_a_causal_mask_and_scales(n):
    w = World(64, 32, FP, 2, [40, 333], seed=n).fill()
    run_attention(w, [n, n], 4, is_causal=False)
    run_attention(w, [n, n], 4, scale=0.0)
    run_attention(w, [n, n], 4, scale=-0.7)
    run_attention(w, [n, n], 4, scale=3.0, lse=False)


@pytest.mark.parametrize("heads,lens", [(1, [5000]), (2, [20000, 1]), (3, [700, 9000, 64])])
def test_attention_of_long_contexts_joined_across_ctas(heads, lens):
    w = World(128, 64, BF, heads, lens, seed=heads).fill()
    run_attention(w, [1] * len(lens), 4 * heads, ragged=False)
    run_attention(w, [min(2, n) for n in lens], 8 * heads)


@pytest.mark.parametrize("rows", [1, 70])
@pytest.mark.parametrize("dtype", [BF, FP])
def test_values_and_scores_of_any_sizes_beside_each_other(rows, dtype):
    """Blocks whose steps lie far apart, seen and not; tokens that weigh next to nothing and are huge."""
    w = World(64, 32, dtype, 1, [400], seed=rows)
    top = 14 if dtype == FP else 38
    for b, e in enumerate([0, -top, top - 2, 0, -3, top // 2, -top // 2, 0, 5, -top, 0, top - 2]):
        w.v[0][16 * b:16 * b + 16] = (w.v[0][16 * b:16 * b + 16].double() * 2.0 ** e / 4).to(dtype)
    w.v[0][16:32] = 0
    w.k[0][48:64] = 0
    w.fill()
    q = w.rand(rows, 4, 64)
    for scale in (0.125, 2.0, -4.0, 1e-6):
        run_attention(w, [rows], 4, scale=scale, q=q)


@pytest.mark.parametrize("rows", [1, 70])
def test_scores_of_2_to_20_and_more(rows):
    """Weights are then one token's, and of tokens with equal keys equal parts."""
    w = World(64, 16, BF, 1, [200], seed=3)
    w.k[0][100:110] = w.k[0][50]
    w.fill()
    k, v = w.stored[0].values()
    q = w.rand(rows, 2, 64)
    q[:, 0] = w.k[0][50, 0]
    for scale in (1e5, 1e8):
        out, _ = run_attention_raw(w, q, scale)
        s = torch.einsum("rhd,ld->rhl", q.double(), k[:, 0]) * scale
        s = s.masked_fill(~causal(rows, 200)[:, None], -math.inf)
        top = s.amax(-1, keepdim=True)
        near = s >= top - top.abs() * 2.0 ** -16  # what fp32 cannot tell apart may get any part
        lo = torch.where(near[..., None], v[None, None, :, 0], torch.full_like(v[None, None, :, 0], math.inf)).amin(2)
        hi = torch.where(near[..., None], v[None, None, :, 0], torch.full_like(v[None, None, :, 0], -math.inf)).amax(2)
        slack = 2.0 ** -7 * torch.maximum(lo.abs(), hi.abs()) + 2.0 ** -20
        assert ((out.double() >= lo - slack) & (out.double() <= hi + slack)).all()


def run_attention_raw(w, q, scale, **kw):
    out, ls = torch.full_like(q, 9.0), torch.full(q.shape[:2], 9.0, device="cuda")
    w.cache.attention(q[None], out[None], scale=scale, lse=ls, **w.batch, **kw)
    return out, ls


@pytest.mark.parametrize("rows", [1, 3, 60])
@pytest.mark.parametrize("side", [0, 1])
def test_tokens_that_are_not_finite(rows, side):
    """Rows that see one are NaN, with NaN keys their lse too; others are what they were; mass takes only finite rows."""
    w = World(128, 32, BF, 2, [100], seed=rows)
    (w.k if side == 0 else w.v)[0][90, 1, 5] = math.inf
    w.fill()
    q = w.rand(rows, 4, 128)
    out, ls = run_attention_raw(w, q, 0.1, weigh=True)
    hit = torch.arange(100 - rows, 100, device="cuda") >= 90
    assert torch.isfinite(out[:, :2]).all() and torch.isnan(out[hit][:, 2:]).all() and torch.isfinite(out[~hit]).all()
    assert torch.isfinite(ls[:, :2]).all() and torch.isfinite(ls[~hit]).all()
    assert torch.isnan(ls[hit][:, 2:]).all() if side == 0 else torch.isfinite(ls).all()
    st = w.stored[0]
    k, v = (torch.where(torch.isnan(x), torch.zeros_like(x), x) for x in st.values())
    want = ref.attention(q, k, v, st.steps()[1], causal(rows, 100), 0.1)
    if side == 0:
        want[2][hit, 2:] = 0  # these rows add nothing
    add, tol = ref.masses(want, 2)
    assert ((w.mass_of(0).double() - add).abs() <= tol + 2.0 ** -23 * add).all()


@pytest.mark.parametrize("rows", [1, 50])
def test_pages_that_are_not_there(rows):
    """Tokens in no page get no weight, and have no mass."""
    w = World(64, 16, FP, 2, [90], seed=rows).fill()
    gone = w.table[0, 2].item()
    w.table[0, 2] = -1
    w.cache.mass.fill_(0.0)
    q = w.rand(rows, 4, 64)
    out, ls = run_attention_raw(w, q, 0.125, weigh=True)
    seen = causal(rows, 90)
    seen[:, 32:48] = False
    st = w.stored[0]
    want = ref.attention(q, *st.values(), st.steps()[1], seen, 0.125)
    ref.check(out, ls, want)
    assert (w.cache.mass[0, gone] == 0).all()
    w.table[0, 2] = gone
    add, tol = ref.masses(want, 2)
    assert ((w.mass_of(0).double() - add).abs() <= tol + 2.0 ** -23 * add).all()


def test_offsets_past_32_bits():
    from moe_expert_layer_sorted_gb300 import KVCache8
    cache = KVCache8.allocate(40000, kv_heads=8, head_dim=128, page_size=64, dtype=BF)
    assert cache.pages.numel() > 1 << 32
    table, lens = ints([[39999, 3, 35001]]), ints([130])
    k, v, q = (torch.randn(1, 130, 8, 128, device="cuda").to(BF) for _ in range(3))
    cache.append(k, v, table=table, lens=lens)
    st = ref.Stored(8, 128).append(k[0], v[0])
    ko, vo = torch.empty_like(k), torch.empty_like(k)
    cache.read(ko, vo, table=table, lens=lens)
    assert same_bits(ko[0], st.values()[0].to(BF)) and same_bits(vo[0], st.values()[1].to(BF))
    for rows in (1, 130):
        x = q[:, -rows:].contiguous()
        out, ls = torch.empty_like(x), torch.empty(rows, 8, device="cuda")
        cache.attention(x, out, table=table, lens=lens, lse=ls, weigh=True)
        ref.check(out[0], ls, ref.attention(x[0], *st.values(), st.steps()[1], causal(rows, 130), 1 / math.sqrt(128)))
    kept = torch.empty(1, 8, 70, dtype=torch.int32, device="cuda")
    masses = torch.cat([cache.mass[0, p] for p in table[0].tolist()], -1)[:, :130].T
    cache.evict(kept, table=table, lens=lens, keep_last=3)
    for h in range(8):
        assert kept[0, h].tolist() == ref.kept(masses[:, h].tolist(), 70, 0, 3)
    st.keep(kept[0].long())
    cache.read(ko[:, :70], vo[:, :70], table=table, lens=ints([70]))
    assert same_bits(ko[0, :70], st.values()[0].to(BF)) and same_bits(vo[0, :70], st.values()[1].to(BF))


def test_strided_queries_and_outputs():
    w = World(64, 32, BF, 2, [77, 30], seed=5).fill()
    for rows in (1, 30):
        packed = torch.randn(2, rows, 12, 64, device="cuda").to(BF)
        q, wide = packed[:, :, 2:10], torch.full((2, rows, 9, 128), 3.0, dtype=BF, device="cuda")
        out = wide[:, :, :8, :64]
        w.cache.attention(q, out, **w.batch)
        for i in range(2):
            ref.check(out[i], None, expected(w, i, q[i].contiguous()))
        assert (wide[:, :, 8] == 3).all() and (wide[..., 64:] == 3).all()


# ------------------------------------------------------------------------ weight of tokens

@pytest.mark.parametrize("D,P,dtype", GEOMETRY)
@pytest.mark.parametrize("per", [1, 4, 7])
def test_weight_of_single_tokens(D, P, dtype, per):
    lens = [1, 2, 15, 16, 17, 64, 129, 257, 0, 1000]
    w = World(D, P, dtype, 2, lens, seed=per).fill()
    for _ in range(2):  # the second time onto the first
        run_attention(w, [1] * len(lens), 2 * per, ragged=False, weigh=True)


@pytest.mark.parametrize("D,P,dtype", GEOMETRY)
@pytest.mark.parametrize("per,counts,extra,is_causal", [(1, [130, 1, 64, 0], [0, 5, 300, 9], True), (4, [33, 200], [100, 0], True),
                                                        (8, [17], [7], False), (3, [129, 40], [0, 1000], True), (5, [3, 2], [70, 0], True)])
def test_weight_of_prompts(D, P, dtype, per, counts, extra, is_causal):
    w = World(D, P, dtype, 2, [a + b for a, b in zip(counts, extra)], seed=per).fill()
    run_attention(w, counts, 2 * per, weigh=True, is_causal=is_causal)


@pytest.mark.parametrize("n", [1, 5, 48])
def test_rows_before_a_sequence_weigh_nothing(n):
    w = World(64, 16, BF, 1, [3, 1, 40, 0], seed=n).fill()
    run_attention(w, [n] * 4, 4, ragged=False, weigh=True)


def test_weights_are_the_same_on_every_run():
    w = World(128, 64, BF, 2, [3000, 700], seed=1).fill()
    for rows in (1, 3, 200):
        q = w.rand(2, rows, 8, 128)
        runs = []
        for _ in range(3):
            w.cache.mass.fill_(0.0)
            out, ls = torch.empty_like(q), torch.empty(2 * rows, 8, device="cuda")
            w.cache.attention(q, out, lse=ls, weigh=True, **w.batch)
            runs.append((out, ls, w.cache.mass.clone()))
        for r in runs[1:]:
            assert all(torch.equal(a, b) for a, b in zip(r, runs[0]))


# ------------------------------------------------------------------------------ eviction

def run_evict(w, budget, first, last, masses):
    for i, m in enumerate(masses):
        w.set_mass(i, m)
    guard, mass = w.cache.pages.clone(), w.cache.mass.clone()
    kept = torch.full((len(w.lens), w.heads, budget), 77, dtype=torch.int32, device="cuda")
    w.cache.evict(kept, keep_first=first, keep_last=last, **w.batch)
    touched = torch.zeros(guard.shape[1], guard.shape[3], dtype=torch.bool, device="cuda")  # (page, block) written to
    for i, n in enumerate(w.lens):
        want = [ref.kept(masses[i][:, h].tolist(), budget, first, last) for h in range(w.heads)]
        got = kept[i].tolist()
        for h in range(w.heads):
            assert got[h] == want[h] + [-1] * (budget - len(want[h])), f"sequence {i}, head {h}"
        if n > budget:
            at = torch.tensor(want, device="cuda")
            w.stored[i].keep(at)
            moved = w.mass_of(i, budget)
            assert same_bits(moved, masses[i].gather(0, at.T))
            for b in range(-(-budget // 16)):
                touched[w.table[i, 16 * b // w.P].long(), 16 * b % w.P // 16] = True
            beyond = w.mass_of(i)[budget:]
            assert same_bits(beyond, masses[i][budget:])  # left as it was
    w.holds([min(n, budget) for n in w.lens])
    assert torch.equal(w.cache.pages[0].transpose(1, 2)[~touched], guard[0].transpose(1, 2)[~touched])
    return kept


@pytest.mark.parametrize("D,P,dtype", GEOMETRY)
@pytest.mark.parametrize("budget,first,last", [(64, 4, 8), (37, 0, 0), (100, 0, 37), (16, 16, 0), (1, 0, 1), (33, 32, 1)])
def test_evict(D, P, dtype, budget, first, last):
    lens = [200, 64, 38, 101, 1, 0, 300]
    w = World(D, P, dtype, 2, lens, seed=budget).fill([40, 7])
    masses = [torch.exp(2 * torch.randn(n, 2, generator=w.g, device="cuda")) for n in lens]
    run_evict(w, budget, first, last, masses)


@pytest.mark.parametrize("kind", ["equal", "zeros", "nan", "few", "signs", "close"])
def test_evict_ties_and_odd_masses(kind):
    """Ties go to the lower position, NaN and -inf below everything."""
    w = World(64, 16, FP, 2, [700, 90], seed=2).fill()
    masses = []
    for n in w.lens:
        m = torch.rand(n, 2, generator=w.g, device="cuda")
        if kind == "equal":
            m = torch.full_like(m, 0.25)
        elif kind == "zeros":
            m = torch.where(m < 0.9, torch.where(m < 0.5, 0.0, -0.0).to(m), m)
        elif kind == "nan":
            m = torch.where(m < 0.4, math.nan, torch.where(m < 0.5, -math.inf, torch.where(m > 0.9, math.inf, m)))
        elif kind == "few":
            m = (m * 4).floor()
        elif kind == "signs":
            m = m - 0.5
        else:  # the last bits alone differ
            m = (torch.full_like(m, 1.5).view(torch.int32) + (m * 40).int()).view(torch.float32)
        masses.append(m)
    run_evict(w, 50, 3, 5, masses)


@pytest.mark.parametrize("heads,lens,budget,first,last", [(1, [70000], 33333, 17, 1000), (2, [9000, 20000], 8192, 0, 64), (8, [5000] * 9, 4096, 4, 100)])
def test_evict_long_sequences(heads, lens, budget, first, last):
    w = World(128, 64, BF, heads, lens, seed=heads).fill()
    masses = [torch.exp(2 * torch.randn(n, heads, generator=w.g, device="cuda")) for n in lens]
    run_evict(w, budget, first, last, masses)


def test_evict_moves_marks_and_keeps_other_layers():
    w = World(128, 32, BF, 2, [100], layers=3, layer=1)
    w.v[0][60, 0, 3], w.k[0][70, 1, 0] = math.nan, math.inf
    w.fill()
    other = w.cache.pages[::2].clone()
    mass = torch.rand(100, 2, generator=w.g, device="cuda")
    mass[[60, 70]] = 9.0
    w.set_mass(0, mass)
    kept = torch.empty(1, 2, 40, dtype=torch.int32, device="cuda")
    w.cache.evict(kept, **w.batch)
    w.stored[0].keep(kept[0].long())
    w.holds([40])
    assert all(torch.isnan(x).any() for x in w.stored[0].values())
    assert torch.equal(other, w.cache.pages[::2])


def test_evict_with_pages_that_are_not_there():
    """Tokens in no page go first; a page that is not there takes nothing."""
    w = World(64, 16, BF, 1, [100], seed=4).fill()
    mass = torch.rand(100, 1, generator=w.g, device="cuda")
    w.set_mass(0, mass)
    w.table[0, 3] = 1 << 20
    mass[48:64] = -math.inf
    kept = torch.empty(1, 1, 70, dtype=torch.int32, device="cuda")
    w.cache.evict(kept, **w.batch)
    assert kept[0, 0].tolist() == ref.kept(mass[:, 0].tolist(), 70, 0, 0)
    w.stored[0].keep(kept[0].long())
    (k,), (v,) = w.read([70])
    there = (torch.arange(70, device="cuda") // 16 != 3) & (kept[0, 0] // 16 != 3)
    for got, want in zip((k, v), w.stored[0].values()):
        assert same_bits(got[there], want[there].float().to(BF))


def test_a_cache_at_a_budget():
    """Prompt, steps, eviction, steps: attention over what is stored, all along, and the mass that decides."""
    w = World(128, 64, BF, 2, [400, 90], seed=7)
    have, w.lens = [300, 40], [300, 40]
    k, v = w.k, w.v
    for i, n in enumerate(have):
        w.stored[i].append(k[i][:n], v[i][:n])
    w.lens_t = ints(have)
    w.cache.append(torch.cat([k[i][:n] for i, n in enumerate(have)]), torch.cat([v[i][:n] for i, n in enumerate(have)]),
                   starts=starts_of(have), max_new=300, **w.batch)
    run_attention(w, have, 8, weigh=True)
    at = list(have)
    for step in range(40):
        for i in range(2):
            w.stored[i].append(k[i][at[i]:at[i] + 1], v[i][at[i]:at[i] + 1])
        new = [x[i][at[i]:at[i] + 1] for x in (k, v) for i in range(2)]
        at = [x + 1 for x in at]
        w.lens = [x + 1 for x in w.lens]
        w.lens_t = ints(w.lens)
        w.cache.append(torch.stack(new[:2]), torch.stack(new[2:]), **w.batch)
        run_attention(w, [1, 1], 8, ragged=False, weigh=True)
        if step % 16 == 15:
            masses = [w.mass_of(i).clone() for i in range(2)]
            run_evict(w, 64, 4, 16, masses)
            w.lens = [min(x, 64) for x in w.lens]
            w.lens_t = ints(w.lens)


# ------------------------------------------------------------------- streams, graphs, refusals

def test_captured_and_replayed():
    """A step (write, attention, weights) and an eviction as one graph, twice."""
    w = World(64, 16, BF, 2, [60, 33], seed=9).fill()
    for i in range(2):
        w.stored[i] = ref.Stored(2, 64)
    k, v, q = w.rand(2, 1, 2, 64), w.rand(2, 1, 2, 64), w.rand(2, 1, 4, 64)
    out, ls, kept = torch.empty_like(q), torch.empty(2, 4, device="cuda"), torch.empty(2, 2, 32, dtype=torch.int32, device="cuda")

    def step():
        w.cache.append(k, v, **w.batch)
        w.cache.attention(q, out, lse=ls, weigh=True, **w.batch)
        w.cache.evict(kept, keep_last=1, **w.batch)

    start = (w.cache.pages.clone(), w.cache.mass.nan_to_num(0.0).clone())
    results = []
    for graph in (False, True, True):
        w.cache.pages.copy_(start[0])
        w.cache.mass.copy_(start[1])
        if not graph:
            step()
        elif len(results) == 1:
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g):
                step()
            g.replay()
        else:
            g.replay()
        torch.cuda.synchronize()
        results.append([x.clone() for x in (out, ls, kept, w.cache.pages, w.cache.mass)])
    w.cache.check()
    for r in results[1:]:
        assert all(torch.equal(a, b) for a, b in zip(r, results[0]))


def test_calls_on_two_streams_share_the_workspace_in_turn():
    w = World(128, 64, BF, 1, [30000], seed=1).fill()
    q = [w.rand(1, 1, 8, 128) for _ in range(8)]
    want = []
    for x in q:
        o = torch.empty_like(x)
        w.cache.attention(x, o, **w.batch)
        want.append(o)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = [torch.empty_like(x) for x in q]
    torch.cuda.synchronize()
    for i, x in enumerate(q):
        w.cache.attention(x, outs[i], stream=streams[i % 2], **w.batch)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(outs, want))


def test_a_wait_that_runs_out_is_reported_and_does_no_lasting_harm():
    from moe_expert_layer_sorted_gb300 import MoeError
    w = World(128, 64, BF, 2, [5000], seed=6).fill()
    q = w.rand(1, 1, 8, 128)
    good, out = torch.empty_like(q), torch.empty_like(q)
    w.cache.attention(q, good, **w.batch)
    w.cache.debug_fail_next_attention()
    w.cache.attention(q, out, **w.batch)
    torch.cuda.synchronize()
    with pytest.raises(MoeError) as e:
        w.cache.check()
    assert e.value.status == 4
    w.cache.attention(q, out, **w.batch)
    torch.cuda.synchronize()
    w.cache.check()
    assert torch.equal(out, good)


def test_refusals():
    from moe_expert_layer_sorted_gb300 import KVCache8, MoeError
    w = World(64, 32, BF, 2, [40], seed=1).fill()
    q, out, ls = w.rand(1, 1, 4, 64), torch.empty(1, 1, 4, 64, dtype=BF, device="cuda"), torch.empty(1, 4, device="cuda")
    k = w.rand(1, 1, 2, 64)
    kept = torch.empty(1, 2, 8, dtype=torch.int32, device="cuda")
    c, b = w.cache, w.batch
    plain = KVCache8.allocate(2, kv_heads=2, head_dim=64, page_size=32, mass=False)
    pb = dict(b, table=ints([[0, 1]]))
    guard = c.pages.clone()
    bad = [lambda: c.attention(q, out, weigh=True, **b), lambda: plain.attention(q, out, lse=ls, weigh=True, **pb),
           lambda: plain.evict(kept, **pb), lambda: c.evict(kept, keep_first=5, keep_last=4, **b),
           lambda: c.evict(kept, keep_first=-1, **b), lambda: c.evict(kept, keep_last=-1, **b), lambda: c.evict(kept[:, :1], **b),
           lambda: c.evict(kept.long(), **b), lambda: c.evict(kept[..., ::2], **b), lambda: c.evict(kept[..., :0], **b),
           lambda: c.evict(kept.cpu(), **b), lambda: c.evict(kept, **dict(b, layer=1)), lambda: c.attention(q, q, **b),
           lambda: c.attention(q[:, :, :3], out[:, :, :3], **b), lambda: c.attention(q.half(), out, **b),
           lambda: c.attention(q, out, scale=math.inf, **b), lambda: c.attention(q, out, lse=ls[:, :2], **b),
           lambda: c.attention(q, out, **dict(b, layer=-1)), lambda: c.append(k, k[:, :, :1], **b), lambda: c.append(k.float(), k, **b),
           lambda: c.append(k, k, **dict(b, lens=w.lens_t.long())), lambda: c.append(k, k, **dict(b, table=w.table[0])),
           lambda: c.read(k, k.expand(1, 1, 2, 64).half(), **b)]
    for i, f in enumerate(bad):
        with pytest.raises(MoeError) as e:
            f()
        assert e.value.status == 1, i
    assert torch.equal(guard, c.pages)
    for kw in (dict(head_dim=96), dict(page_size=48), dict(page_size=8), dict(kv_heads=1025), dict(dtype=torch.float32)):
        with pytest.raises(MoeError):
            KVCache8.allocate(2, **dict(dict(kv_heads=2, head_dim=64, page_size=32), **kw))
    c.evict(kept[:0], table=w.table[:0], lens=w.lens_t[:0])  # no sequences: nothing to do
    c.close()
    with pytest.raises(MoeError, match="closed"):
        c.check()


def test_a_wait_of_a_prompt_that_runs_out_is_reported():
    from moe_expert_layer_sorted_gb300 import MoeError
    w = World(128, 64, BF, 2, [700], seed=6).fill()
    q = w.rand(1, 300, 4, 128)
    good, out = torch.empty_like(q), torch.empty_like(q)
    w.cache.attention(q, good, **w.batch)
    w.cache.debug_fail_next_attention()
    w.cache.attention(q, out, **w.batch)
    torch.cuda.synchronize()
    with pytest.raises(MoeError) as e:
        w.cache.check()
    assert e.value.status == 4
    w.cache.attention(q, out, **w.batch)
    torch.cuda.synchronize()
    w.cache.check()
    assert torch.equal(out, good)


@pytest.mark.parametrize("rows", [1, 4, 90])
@pytest.mark.parametrize("dtype", [BF, FP])
def test_queries_that_are_not_finite_harm_no_other_row(rows, dtype):
    """A query row and head with an infinity or a NaN is NaN and weighs nothing; the others are what they were, within
    each row's own bound (not to the bit: 32 rows share the moments at which their references rise, and whichever these
    are, a row is within its bound of the exact value)."""
    w = World(64, 16, dtype, 2, [150], seed=rows).fill()
    q = w.rand(rows, 8, 64)
    bad = q.clone()
    hit = torch.zeros(rows, 8, dtype=torch.bool, device="cuda")
    for r, h, x in ((0, 1, math.nan), (rows - 1, 6, math.inf), (rows // 2, 5, -math.inf)):
        bad[r, h, 7] = x
        hit[r, h] = True
    out, ls = run_attention_raw(w, bad, 0.125, weigh=True)
    assert torch.isnan(out[hit]).all() and not torch.isfinite(ls[hit]).any()
    full = expected(w, 0, q, 0.125)
    ref.check(out[~hit], ls[~hit], [x[~hit] for x in full])
    full[2][hit] = 0
    add, tol = ref.masses(full, 2)
    assert ((w.mass_of(0).double() - add).abs() <= tol + 2.0 ** -23 * add).all()


@pytest.mark.parametrize("rows,lens", [(1, [70, 0, 33]), (5, [70, 0, 33]), (64, [130, 0, 64])])
def test_weights_without_room_for_scores(rows, lens):
    """A table of so many pages that scores would not fit the workspace: made again from the keys, the same sums."""
    w = World(64, 256, BF, 4, lens, seed=rows).fill()
    wide = torch.full((3, 1 << 15), -1, dtype=torch.int32, device="cuda")  # 8,388,608 tokens a sequence
    wide[:, :w.cols] = w.table
    w.table = wide
    run_attention(w, [rows] * 3, 8, ragged=False, weigh=True)


def test_tables_with_strides_and_lengths_beyond_them():
    """Rows of a wider table; lens larger than its pages hold: what is there counts, in every call."""
    w = World(64, 16, BF, 2, [64, 50], seed=2).fill()
    wide = torch.full((2, 9), 1 << 29, dtype=torch.int32, device="cuda")
    wide[:, 2:2 + w.cols] = w.table
    w.table = wide[:, 2:2 + w.cols]
    q = w.rand(2, 1, 4, 64)
    out, ls = torch.empty_like(q), torch.empty(2, 4, device="cuda")
    w.cache.attention(q, out, table=w.table, lens=w.lens_t, lse=ls, weigh=True)
    for i in range(2):
        ref.check(out[i], ls[i:i + 1], expected(w, i, q[i]))
    w.lens_t = ints([1000, 50])
    kept = torch.empty(2, 2, 40, dtype=torch.int32, device="cuda")
    masses = [w.mass_of(i).clone() for i in range(2)]
    w.cache.evict(kept, keep_first=1, keep_last=2, **w.batch)
    for i, n in enumerate((64, 50)):
        for h in range(2):
            assert kept[i, h].tolist() == ref.kept(masses[i][:n, h].tolist(), 40, 1, 2)
        w.stored[i].keep(kept[i].long())
    w.holds([40, 40])


@pytest.mark.parametrize("dtype", [BF, FP])
def test_turned_codes_at_every_ratio_of_steps(dtype):
    """Steps whose ratios are simple fractions (quotients near and on halves), powers of two, near one and tiny: codes
    moved by an eviction, and older codes of a block that grows."""
    n = 16 * 40
    w = World(64, 16, dtype, 1, [n], seed=1)
    codes = torch.arange(-127, 128, device="cuda", dtype=torch.float64)
    g = torch.Generator(device="cuda").manual_seed(5)
    tops = [127.0, 254.0, 96.0, 192.0, 160.0, 200.0, 128.0, 64.0, 255.0, 253.0, 129.0, 1.0, 0.5, 3.0, 5.0, 6.0, 7.0, 9.0, 2.0 ** -10, 0.0]
    x = torch.empty(n, 64, dtype=torch.float64, device="cuda")
    for b in range(40):
        top = tops[b % len(tops)]
        pick = codes[torch.randint(0, 255, (16, 64), generator=g, device="cuda")] * (top / 127)
        pick[0, 0] = top
        x[16 * b:16 * b + 16] = pick
    w.k[0] = x[:, None].to(dtype)
    w.v[0] = x.flip(0)[:, None].to(dtype).contiguous()
    w.fill([3, 5])
    w.holds()
    mass = torch.rand(n, 1, generator=g, device="cuda")
    run_evict(w, 200, 0, 0, [mass])
    w.lens, w.lens_t = [200], ints([200])
    run_evict(w, 77, 1, 1, [mass[:200].contiguous()])


def test_weights_of_sequences_with_and_without_room_for_scores():
    """The workspace holds the scores of 16,256 rounds of 128 tokens at 16 columns: the first sequence's, not the others'."""
    w = World(64, 64, BF, 64, [9000, 0, 9000, 300], seed=5).fill()
    run_attention(w, [8] * 4, 256, ragged=False, weigh=True)


@pytest.mark.parametrize("rows", [1, 9])
def test_weights_of_many_sequences_of_one_much_longer(rows):
    """More sequences than a CTA has threads; a CTA that takes several stretches of one sequence's scores; a table far wider
    than most of them."""
    lens = [int(n) for n in torch.randint(0, 40, (300,), generator=torch.Generator().manual_seed(rows))]
    lens[257] = 5000
    w = World(64, 16, FP, 8, lens, seed=rows).fill()
    w.cache.mass.nan_to_num_(0.25)
    run_attention(w, [rows] * 300, 32, ragged=False, weigh=True)


@pytest.mark.parametrize("counts", [[300, 0, 1, 40], [1, 40, 700, 0], [33, 33, 33, 33]])
@pytest.mark.parametrize("is_causal", [True, False])
def test_weights_of_uneven_prompts_in_wide_tables(counts, is_causal):
    """Work of all sizes cut into equal shares: sequences without rows or tokens, rows before their sequence."""
    w = World(128, 64, BF, 3, [900, 20, 690, 0], seed=sum(counts)).fill()
    wide = torch.full((4, 2048), -1, dtype=torch.int32, device="cuda")
    wide[:, :w.cols] = w.table
    w.table = wide
    run_attention(w, counts, 15, weigh=True, is_causal=is_causal)


@pytest.mark.parametrize("heads,lens,budget", [(8, [700, 0, 273, 272] * 8, 272), (4, [3000, 2500, 2100, 1999, 4000], 2000)])
def test_evict_in_clusters_of_other_sizes(heads, lens, budget):
    """More clusters than run at once; clusters of a number of CTAs that is no power of two.  Blocks of far steps, marks."""
    w = World(64, 32, FP, heads, lens, seed=budget)
    for k, v in zip(w.k, w.v):
        n = len(k)
        far = torch.exp2(torch.randint(-6, 3, (-(-n // 16), 1, 1), generator=w.g, device="cuda").float())
        far = far.repeat_interleave(16, 0)[:n]
        k.copy_((k.float() * far).to(k.dtype))
        v.copy_((v.float() * far.flip(0)).to(v.dtype))
        k[5::97] = math.nan
        v[11::89, ..., 3] = math.inf
    w.fill()
    masses = [torch.exp(2 * torch.randn(n, heads, generator=w.g, device="cuda")) for n in lens]
    run_evict(w, budget, 4, 50, masses)


def test_first_calls_of_a_cache_are_captured():
    """Nothing that a cache does once is in the way of a capture."""
    w = World(64, 64, BF, 4, [1500, 900], seed=7).fill()
    masses = [torch.rand(n, 4, generator=w.g, device="cuda") for n in w.lens]
    for i, m in enumerate(masses):
        w.set_mass(i, m)
    kept = torch.empty(2, 4, 1000, dtype=torch.int32, device="cuda")
    q = w.rand(2, 1, 8, 64)
    out, ls = torch.empty_like(q), torch.empty(2, 8, device="cuda")
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        w.cache.attention(q, out, lse=ls, weigh=True, **w.batch)
        w.cache.evict(kept, keep_first=4, keep_last=16, **w.batch)
    graph.replay()
    torch.cuda.synchronize()
    for i in range(2):
        want = expected(w, i, q[i])
        ref.check(out[i], ls[i:i + 1], want)
        n = w.lens[i]
        assert (kept[i, :, :min(n, 1000)].diff(dim=1) > 0).all() and (kept[i, :, n:] == -1).all()
        if n > 1000:
            w.stored[i].keep(kept[i].long())
    w.holds([1000, 900])


@pytest.mark.parametrize("rows", [1, 40])
def test_rows_beyond_fp32_weigh_nothing(rows):
    """A scale that takes every score out of fp32's range: no row is finite, and mass stays what it was."""
    w = World(64, 64, BF, 2, [130], seed=rows).fill()
    out, ls = run_attention_raw(w, w.rand(rows, 4, 64), 3e38, weigh=True)
    assert not torch.isfinite(ls).any()
    assert (w.mass_of(0) == 0).all()
