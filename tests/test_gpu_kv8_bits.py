"""The 8-bit cache's weights in 16 bits: tokens of little weight beside some of much weight whose values are nothing, so
that the little ones make up the result."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

BF, FP = torch.bfloat16, torch.float16
HALF = {BF: 2.0 ** -8, FP: 2.0 ** -11}  # half a step, relative


def cache_of(level, v, heads, dtype, D=64, P=64, far=None):
    """Tokens whose scores are their `level` (whole numbers up to 127) times the queries' first channel, and whose
    values v [N, D] are whole numbers of 0..127, all of them stored as they are (127 in every block: steps of 1).  far: the
    keys' third channel."""
    from moe_expert_layer_sorted_gb300 import KVCache8
    n = len(level)
    cache = KVCache8.allocate(-(-n // P), kv_heads=heads, head_dim=D, page_size=P, dtype=dtype)
    k = torch.zeros(n, D, device="cuda")
    k[:, 0], k[:, 1] = level.float(), 127.0
    if far is not None:
        k[:, 2] = far
    v = v.clone()
    v[15::16, 0] = 127.0
    table = torch.arange(-(-n // P), dtype=torch.int32, device="cuda")[None]
    rows = [x.to(dtype)[None, :, None].expand(1, n, heads, D).contiguous() for x in (k, v)]
    cache.append(*rows, table=table, lens=torch.tensor([n], dtype=torch.int32, device="cuda"))
    back = [torch.empty_like(x) for x in rows]
    cache.read(*back, table=table, lens=torch.tensor([n], dtype=torch.int32, device="cuda"))
    assert torch.equal(back[0], rows[0]) and torch.equal(back[1], rows[1])
    return cache, table, v.double()


def wanted(y, v, tile, first, other):
    """Result of weights 2^y over values v >= 0 in 64 bits, and how far it may be off.  All steps are 1.  A weight enters
    with 11 bits, or is off by `other` of its tile's (`tile` tokens) sum or largest, or by `first` of the largest where that is
    the largest so far; by no more than itself.  (Scores are exact up to 2^-22 of them, exponentials to 2^-22.)"""
    p = torch.exp2(y - y.max()).double()
    pad = torch.cat((p, p.new_zeros(-len(p) % tile))).view(-1, tile)
    most = pad.amax(1)
    so_far = torch.cat((most.new_zeros(1), most.cummax(0).values[:-1]))
    unit = pad.sum(1) if tile == 128 else most
    floor = torch.where(most >= so_far, first * most, other * unit)
    off = pad * (2.0 ** -11 + 2.0 ** -15) + torch.minimum(floor[:, None], pad)
    out = p @ v
    return out / p.sum(), (off.flatten()[:len(p)] @ v) / p.sum()


def run(cache, table, v, level, unit, rows, per, batch, dtype):
    """Rows whose scores are level times unit, three quarters and a half of it, in log2 units."""
    heads, D = cache.kv_heads, cache.head_dim
    share = torch.tensor([1.0, 0.75, 0.5])
    q = torch.zeros(batch, rows, heads * per, D, device="cuda")
    pick = torch.arange(batch * rows * heads * per).view(batch, rows, heads * per) % 3
    q[..., 0] = share[pick].cuda()
    out = torch.empty(q.shape, dtype=dtype, device="cuda")
    cache.attention(q.to(dtype), out, table=table.expand(batch, -1).contiguous(), causal=False, scale=unit * math.log(2),
                    lens=torch.full((batch,), len(level), dtype=torch.int32, device="cuda"))
    few = rows * per <= 32
    for i, s in enumerate(share.tolist()):
        want, tol = wanted(level.double() * unit * s, v, *((16, 2.0 ** -25, 2.0 ** -17) if few else (128, 2.0 ** -27, 2.0 ** -19)))
        tol = tol + HALF[dtype] * want * 1.01 + (2.0 ** -24 if dtype == FP else 0.0)
        got = out[pick.cuda() == i].double()
        off = ((got - want).abs() / tol).max().item()
        assert off <= 1, f"{s}: {off} of the bound, {((got - want).abs().norm() / want.norm() / len(got) ** 0.5).item():.1e} of the result"


# 320 items of single tokens, so that one CTA takes the whole of most; 80 pairs of row tiles, so that none is cut
FEW, MANY = dict(rows=1, per=4, batch=40), dict(rows=640, per=4, batch=1)


@pytest.mark.parametrize("shape", [FEW, MANY], ids=["few", "many"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("apart,dtype", [(12.0, FP), (18.3, FP), (20.9, FP), (22.912, FP), (30.2, BF), (41.7, BF), (52.0, BF)])
def test_one_token_of_much_weight_and_no_value(shape, D, apart, dtype):
    n = 16384
    gen = torch.Generator(device="cuda").manual_seed(1)
    v = torch.randint(64, 128, (n, D), generator=gen, device="cuda").float()
    level = torch.zeros(n, dtype=torch.int32, device="cuda")
    level[3] = 127
    v[3] = 0
    cache, table, v = cache_of(level, v, 8, dtype, D)
    run(cache, table, v, level, apart / 127, dtype=dtype, **shape)


@pytest.mark.parametrize("shape", [FEW, MANY], ids=["few", "many"])
@pytest.mark.parametrize("order", ["down", "up", "both", "last"])
def test_weights_that_fall_and_rise(shape, order):
    """Steps of 2^-9.4 and less every 256 tokens, values in the lightest steps alone; the same upwards, and down and up."""
    steps, each = 6, 256
    gen = torch.Generator(device="cuda").manual_seed(2)
    down = torch.arange(steps - 1, -1, -1, device="cuda").repeat_interleave(each)
    stairs = {"down": down, "up": down.flip(0), "both": torch.cat((down, down.flip(0), down)),
              "last": torch.cat((down.new_zeros(2048), down.new_full((1,), 5), down.new_zeros(2047)))}[order]
    v = torch.randint(64, 128, (len(stairs), 64), generator=gen, device="cuda").float()
    v[stairs > 0] = 0
    cache, table, v = cache_of(25 * stairs.int(), v, 8, BF)
    run(cache, table, v, 25 * stairs.int(), 9.4 / 25, dtype=BF, **shape)


def test_weights_that_fall_where_another_row_rises_far():
    """Rows that share a warp: of some, the second 128 tokens are little beside the first one (which has no value); of the
    others, they are 2^70 of all before."""
    n, rows, per, unit = 384, 640, 4, 22.912 / 127
    gen = torch.Generator(device="cuda").manual_seed(3)
    v = torch.randint(64, 128, (n, 64), generator=gen, device="cuda").float()
    level = torch.zeros(n, dtype=torch.int32, device="cuda")
    level[3] = 127
    v[3] = 0
    far = torch.zeros(n, device="cuda")
    far[128:] = 127
    cache, table, v = cache_of(level, v, 8, FP, far=far)
    q = torch.zeros(1, rows, 8 * per, 64, device="cuda")
    q[:, :, ::2, 0] = 1
    q[:, :, 1::2, 2] = 70 / 22.912
    q = q.to(FP)
    out = torch.empty_like(q)
    cache.attention(q, out, table=table, causal=False, scale=unit * math.log(2), lens=torch.tensor([n], dtype=torch.int32, device="cuda"))
    for h, y in ((0, level.double() * unit), (1, far.double() * unit * q[0, 0, 1, 2].double())):
        want, tol = wanted(y, v, 128, 2.0 ** -27, 2.0 ** -17)
        off = ((out[0, -n:, h::2].double() - want).abs() / (tol + 1.01 * HALF[FP] * want + 2.0 ** -24)).max().item()
        assert off <= 1, (h, off)
    assert (out[0, :-n] == 0).all()  # rows before the first token
