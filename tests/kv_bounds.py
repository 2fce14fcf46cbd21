"""Attention in 64 bits with an error bound per row and channel from what that row sees."""
import math

import torch

import kv_reference as ref


def attention(q, k, v, seen, scale, group):
    """q [R, Hq, D] 16-bit, k, v [L, H, D] in 64 bits, in groups of `group` channels, seen [R, L] bool -> out, lse and their bounds.

    A score is off by at most ds, 2^-11 for keys rounded to fp16 (half a unit in the last place of
    11 bits, relative to a number just above a power of two) and 2^-16 for fp32 sums, times its
    terms' magnitude; a weight by twice that, relatively; weights
    (times steps) and values are rounded once each to 11 bits.  So a channel is off by that part
    of sum p |v|, with |v| up to the largest stored value of its group (codes are what is
    multiplied, so a small value of a group carries the group's rounding), and by the output's
    own rounding."""
    u16 = 2.0 ** -11
    u = ref.UNIT[q.dtype]
    R, Hq, D = q.shape
    L, H, _ = k.shape
    qd = q.double().view(R, H, Hq // H, D)
    seen = seen[:, None, None, :]
    s = torch.einsum("rhgd,lhd->rhgl", qd, k) * scale
    mag = torch.einsum("rhgd,lhd->rhgl", qd.abs(), k.abs()) * abs(scale)
    s = s.masked_fill(~seen, -math.inf)
    top = s.amax(-1, keepdim=True)
    p = torch.exp(s - torch.where(torch.isfinite(top), top, torch.zeros_like(top)))
    tot = p.sum(-1, keepdim=True)
    p = p / tot.clamp_min(1e-300)
    lse = torch.where(tot[..., 0] > 0, top[..., 0] + torch.log(tot[..., 0].clamp_min(1e-300)), top[..., 0])
    out = torch.einsum("rhgl,lhd->rhgd", p, v)
    ds = torch.where(seen & (p > 2.0 ** -60), mag, torch.zeros_like(mag)).amax(-1) * (u16 + 2.0 ** -16) + 2.0 ** -16
    big = v.abs().unflatten(-1, (-1, group)).amax(-1, keepdim=True).expand(L, H, D // group, group).flatten(2)
    terms = torch.einsum("rhgl,lhd->rhgd", p, big)
    tol = (2.2 * ds + 2.0 ** -9)[..., None] * terms + 1.1 * u * out.abs() + 2.0 ** -134
    if q.dtype == torch.float16:
        tol = tol + 2.0 ** -24
    return out.flatten(1, 2), lse.flatten(1, 2), tol.flatten(1, 2), (1.1 * ds + 2.0 ** -18 * lse.abs().nan_to_num(0, 0, 0)).flatten(1, 2)


def causal(n, L, device="cuda"):
    return torch.arange(L, device=device)[None] <= torch.arange(L - n, L, device=device)[:, None]


def check(out, lse, want, what=""):
    o, ls, tol, ltol = want
    assert torch.isfinite(out).all(), what
    off = (out.double() - o).abs() / tol
    assert (off <= 1).all(), f"{what}: {float(off.max())} of the bound at {(off == off.max()).nonzero()[0].tolist()}"
    if lse is not None:
        empty = torch.isinf(ls)
        assert (lse[empty] == -math.inf).all(), what
        assert ((lse.double() - ls)[~empty].abs() <= ltol[~empty] + 1e-5).all(), what
