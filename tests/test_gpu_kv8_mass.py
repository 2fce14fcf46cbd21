"""Attention over the 8-bit cache with queries and keys of far sizes, and what it adds to the mass of its tokens."""
import pytest
import torch

import kv8_reference as ref
from test_gpu_kv8 import BF, World, causal, expected, ints, run_attention, run_attention_raw

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


@pytest.mark.parametrize("rows", [1, 4, 300])
def test_a_wait_that_runs_out_leaves_no_mass_that_is_wrong(rows):
    """Rows of what gave up are NaN and add nothing; those of the rest add what they do; and the next call is right."""
    from moe_expert_layer_sorted_gb300 import MoeError
    w = World(128, 64, BF, 2, [5000], seed=6).fill()
    q = w.rand(1, rows, 8, 128)
    good, out, ls = torch.empty_like(q), torch.empty_like(q), torch.empty(rows, 8, device="cuda")

    def call(to):
        w.cache.mass.fill_(0.5)
        w.cache.attention(q, to, lse=ls, weigh=True, **w.batch)
        torch.cuda.synchronize()
        return w.mass_of(0).clone()

    mass = call(good)
    # scores of an earlier call lie in the workspace that are much larger than these
    w.cache.attention(w.rand(1, 1, 8, 128), torch.empty(1, 1, 8, 128, dtype=BF, device="cuda"), scale=1e4, weigh=True,
                      lse=torch.empty(1, 8, device="cuda"), **w.batch)
    w.cache.debug_fail_next_attention()
    late = call(out)
    with pytest.raises(MoeError) as e:
        w.cache.check()
    assert e.value.status == 4
    lost = torch.isnan(out[0]).any(-1)
    assert lost.any() and torch.isnan(out[0][lost]).all() and torch.equal(torch.isnan(ls), lost)
    assert torch.equal(out[0][~lost], good[0][~lost])
    assert (late >= 0.5).all() and (late <= mass * (1 + 2.0 ** -20)).all()
    assert torch.equal(call(out), mass) and torch.equal(out, good)
    w.cache.check()


@pytest.mark.parametrize("rows", [40, 2000])
def test_a_wait_of_the_weighing_that_runs_out_is_reported(rows):
    """The first tokens of the first head get nothing then, the others all that they should or less; the next call is right."""
    from moe_expert_layer_sorted_gb300 import MoeError
    w = World(64, 64, BF, 2, [5000], seed=7).fill()
    q = w.rand(1, rows, 8, 64)
    out, ls = torch.empty_like(q), torch.empty(rows, 8, device="cuda")

    def call():
        w.cache.mass.fill_(0.5)
        w.cache.attention(q, out, lse=ls, weigh=True, **w.batch)
        torch.cuda.synchronize()
        return w.mass_of(0).clone()

    mass = call()
    assert (mass > 0.5).all()
    w.cache.debug_fail_next_attention()
    late = call()
    with pytest.raises(MoeError) as e:
        w.cache.check()
    assert e.value.status == 4
    assert (late[:256, 0] == 0.5).all() and (late >= 0.5).all() and (late <= mass * (1 + 2.0 ** -20)).all()
    assert torch.equal(late[:, 1], mass[:, 1])
    assert torch.equal(call(), mass)
    w.cache.check()


@pytest.mark.parametrize("rows", [1, 5, 70])
@pytest.mark.parametrize("scale", [2.0 ** 10, 2.0 ** 14, 1e5, 1e8])
def test_every_row_adds_one_in_all(rows, scale):
    """Weights are those that the attention itself uses, so that each row's sum to 1 whatever the size of its scores:
    up to the exponentials (2^-22), the two sums of up to 200 terms and the quotient, 2^-15 in all."""
    w = World(64, 16, BF, 1, [200], seed=3)
    w.k[0][100:110] = w.k[0][50]
    w.fill()
    w.cache.mass.fill_(0.0)
    q = w.rand(rows, 4, 64)
    q[:, 0] = w.k[0][50, 0]
    _, ls = run_attention_raw(w, q, scale, weigh=True)
    assert torch.isfinite(ls).all()
    assert abs(w.mass_of(0).double().sum().item() - 4 * rows) <= 4 * rows * 2.0 ** -15


@pytest.mark.parametrize("rows", [1, 40])
@pytest.mark.parametrize("score", [2.0 ** 13, 2.0 ** 18, 2.0 ** 20, 2.0 ** 24])
def test_a_row_that_sees_one_token_gives_it_a_weight_of_one(rows, score):
    """40 sequences of a token each (in one call with longer ones, so that the kernels take many rows)."""
    counts = [1] * 8 + [rows]
    w = World(64, 16, BF, 1, [1] * 8 + [rows], seed=rows).fill()
    w.cache.mass.fill_(0.0)
    q = w.rand(sum(counts), 4, 64)
    s = [abs(float(torch.einsum("hd,d->h", q[i].double(), w.stored[i].values()[0][0, 0]).abs().max())) for i in range(8)]
    out, ls = torch.empty_like(q), torch.empty(len(q), 4, device="cuda")
    starts = ints([sum(counts[:i]) for i in range(10)])
    w.cache.attention(q, out, scale=score / max(s), lse=ls, weigh=True, starts=starts, max_new=rows, **w.batch)
    for i in range(8):
        assert abs(w.mass_of(i).item() - 4) <= 4 * 2.0 ** -20, (i, w.mass_of(i).item())


def test_more_rows_than_the_workspace_has_room_for():
    """Rows times heads beyond 2^24: the weights of the later rows are counted from lse itself."""
    from moe_expert_layer_sorted_gb300 import KVCache8
    heads, per, rows, batch, L = 2, 64, 34, 3900, 34  # 16,972,800 of them
    cache = KVCache8.allocate(1, kv_heads=heads, head_dim=64, page_size=64, dtype=BF)
    gen = torch.Generator(device="cuda").manual_seed(1)
    k, v = (torch.randn(1, L, heads, 64, generator=gen, device="cuda").to(BF) for _ in range(2))
    one = torch.zeros(1, 1, dtype=torch.int32, device="cuda")
    cache.append(k, v, table=one, lens=ints([L]))
    st = ref.Stored(heads, 64).append(k[0], v[0])
    # all sequences but the last few have no tokens: nothing of theirs is seen
    lens = torch.zeros(batch, dtype=torch.int32, device="cuda")
    lens[-1] = L
    q = torch.randn(rows, heads * per, 64, generator=gen, device="cuda").to(BF)
    every = torch.zeros(batch, rows, heads * per, 64, dtype=BF, device="cuda")
    every[-1] = q
    out, ls = torch.empty_like(every), torch.empty(batch * rows, heads * per, device="cuda")
    assert ls.numel() > 1 << 24
    cache.mass.fill_(0.0)
    cache.attention(every, out, table=one.expand(batch, 1).contiguous(), lens=lens, lse=ls, weigh=True)
    want = ref.attention(q, *st.values(), st.steps()[1], causal(rows, L), 1 / 8)
    ref.check(out[-1], ls[-rows:], want)
    add, tol = ref.masses(want, heads)
    assert ((cache.mass[0, 0, :, :L].T.double() - add).abs() <= tol + 2.0 ** -23 * add).all()
    assert (out[:-1] == 0).all()


def test_references_of_more_heads_than_lie_beside_the_parts():
    """More than 2^21 single tokens' rows times heads: their references take some of the scores' room."""
    heads, per, batch = 2, 32, 33000
    w = World(64, 16, BF, heads, [20, 40, 0, 33], seed=2).fill()
    q = w.rand(batch, 1, heads * per, 64)
    table = torch.full((batch, w.cols), -1, dtype=torch.int32, device="cuda")
    lens = torch.zeros(batch, dtype=torch.int32, device="cuda")
    at = [0, 17, 1000, batch - 1]
    table[at], lens[at] = w.table, w.lens_t
    out, ls = torch.empty_like(q), torch.empty(batch, heads * per, device="cuda")
    w.cache.mass.fill_(0.0)
    w.cache.attention(q, out, lse=ls, weigh=True, table=table, lens=lens)
    for i, s in enumerate(at):
        want = expected(w, i, q[s])
        ref.check(out[s], ls[s:s + 1], want)
        add, tol = ref.masses(want, heads)
        assert ((w.mass_of(i).double() - add).abs() <= tol + 2.0 ** -23 * add).all()
