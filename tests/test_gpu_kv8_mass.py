"""Attention over the 8-bit cache with queries and keys of far sizes, and what it adds to the mass of its tokens."""
import pytest
import torch

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
