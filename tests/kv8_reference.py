"""Plain implementation of the 8-bit key/value cache for the tests: what is stored, token by token
in 64 bits from the definition, attention with an error bound per row and channel, weights, and
which tokens an eviction keeps."""
import math

import numpy as np
import torch

HALF = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}  # half a step, relative


def nearest(num, den):
    """num / den to the nearest whole number, ties to even; 0 where den is 0.  (Operands of up to 33 and 24
    bits: a quotient that is not a tie is further from it than 64-bit division rounds.)"""
    return torch.where(den > 0, (num / torch.where(den > 0, den, torch.ones_like(den))).round(), torch.zeros_like(num))


def step_of(x):
    """Step of finite x [..., n] in 64 bits: max |x| / 127 rounded to fp32."""
    return (x.abs().amax(-1) / 127).float().double()


class Stored:
    """The keys and values of one sequence as stored: codes u [2, L, H, D], steps s [2, blocks, H],
    marks [2, L, H]."""

    def __init__(self, heads, dim, device="cuda"):
        self.u = torch.zeros(2, 0, heads, dim, dtype=torch.float64, device=device)
        self.s = torch.zeros(2, 0, heads, dtype=torch.float64, device=device)
        self.bad = torch.zeros(2, 0, heads, dtype=torch.bool, device=device)

    @property
    def length(self):
        return self.u.shape[1]

    def append(self, k, v):
        """k, v [n, H, D], one call's rows."""
        x = torch.stack((k, v)).double()
        bad = ~torch.isfinite(x).all(-1)
        x = torch.where(bad[..., None], torch.zeros_like(x), x)
        old, n = self.length, self.length + x.shape[1]
        blocks = -(-n // 16)
        u = torch.cat((self.u, torch.zeros_like(x)), 1)
        s = torch.cat((self.s, self.s.new_zeros(2, blocks - self.s.shape[1], self.s.shape[2])), 1)
        for b in range(old // 16, blocks):
            lo, hi = max(old, 16 * b), min(n, 16 * b + 16)
            new = x[:, lo - old:hi - old]
            fresh = step_of(new.permute(0, 2, 1, 3).flatten(2))
            was = s[:, b].clone()
            s[:, b] = torch.maximum(fresh, was)
            to = s[:, b][:, None, :, None]
            if lo > 16 * b:
                older = u[:, 16 * b:lo]
                u[:, 16 * b:lo] = torch.where(was[:, None, :, None] < to, nearest(older * was[:, None, :, None], to.expand_as(older)), older)
            u[:, lo:hi] = nearest(new, to.expand_as(new)).clamp(-127, 127)
        self.u, self.s, self.bad = u, s, torch.cat((self.bad, bad), 1)
        return self

    def steps(self):
        """[2, L, H]: every token's step."""
        return self.s.repeat_interleave(16, 1)[:, :self.length]

    def values(self):
        """K, V [L, H, D]."""
        x = self.u * self.steps()[..., None]
        return torch.where(self.bad[..., None], torch.full_like(x, math.nan), x)

    def keep(self, kept):
        """kept [H, n]: the positions that stay."""
        h = torch.arange(kept.shape[0], device=kept.device)[:, None]
        u = self.u[:, kept, h].transpose(1, 2)
        s, bad = self.steps()[:, kept, h].transpose(1, 2), self.bad[:, kept, h].transpose(1, 2)
        n = kept.shape[1]
        pad = torch.cat((s, s.new_zeros(2, -n % 16, s.shape[2])), 1)
        to = pad.unflatten(1, (-1, 16)).amax(2)
        each = to.repeat_interleave(16, 1)[:, :n]
        self.u = torch.where((s == each)[..., None], u, nearest(u * s[..., None], each[..., None].expand_as(u)))
        self.s, self.bad = to, bad
        return self


def block_bytes(block, D):
    """One block's bytes (numpy uint8) -> codes [2, 16, D], steps [2], marks [2, 16], by the layout as documented."""
    k, v = block[:16 * D].reshape(16, D // 16, 16), block[16 * D:32 * D].reshape(8, D // 8, 8, 2)
    u = np.zeros((2, 16, D), np.int64)
    for t in range(16):
        for i in range(D // 16):
            u[0, t, 16 * i:16 * i + 16] = k[t, i ^ (4 * (t & 1)) if D == 128 else i].astype(np.int64) - 128
        p = t // 2
        for i in range(D // 8):
            u[1, t, 8 * i:8 * i + 8] = v[p, i ^ ((p & 1) | (p & 2) << 1) if D == 128 else i ^ (2 * (p & 3)), :, t & 1].astype(np.int64) - 128
    par = block[32 * D:]
    marks = par[8:12].view(np.uint16)
    return u, par[:8].view(np.float32), (marks[:, None] >> np.arange(16)) & 1 > 0


def attention(q, k, v, sv, seen, scale):
    """q [R, Hq, D] 16-bit, k, v [L, H, D] stored values in 64 bits (finite), sv [L, H] the values' steps, seen
    [R, L] bool -> out, lse, weights p [R, Hq, L], and bounds of the first two and, relative, of the weights.

    A score is off by ds: fp32 sums of D products (2^-18 of their magnitude) and the factors' and
    exponents' roundings (2^-16 absolute); so a weight by 2.2 ds, relatively.  A weight times its
    token's step enters with 11 bits (half a step: 2^-11), or, below 2^-14 of the row's largest,
    off by 2^-25 of that largest, times a code of up to 127; the output is rounded once."""
    R, Hq, D = q.shape
    L, H, _ = k.shape
    qd = q.double().view(R, H, Hq // H, D)
    see = seen[:, None, None, :]
    s = torch.einsum("rhgd,lhd->rhgl", qd, k) * scale
    mag = torch.einsum("rhgd,lhd->rhgl", qd.abs(), k.abs()) * abs(scale)
    s = s.masked_fill(~see, -math.inf)
    top = s.amax(-1, keepdim=True) if L else s.new_full(s.shape[:-1] + (1,), -math.inf)
    p = torch.exp(s - torch.where(torch.isfinite(top), top, torch.zeros_like(top)))
    tot = p.sum(-1, keepdim=True)
    p = p / tot.clamp_min(1e-300)
    lse = torch.where(tot[..., 0] > 0, top[..., 0] + torch.log(tot[..., 0].clamp_min(1e-300)), top[..., 0])
    out = torch.einsum("rhgl,lhd->rhgd", p, v)
    counts = see & (p > 2.0 ** -60)
    ds = (torch.where(counts, mag, torch.zeros_like(mag)).amax(-1) if L else mag.sum(-1)) * 2.0 ** -18 + 2.0 ** -16
    ps = p * sv.T[None, :, None, :]
    most = ps.amax(-1) if L else ps.sum(-1)
    small = (see & (ps < most[..., None] * 2.0 ** -14)).sum(-1)
    terms = torch.einsum("rhgl,lhd->rhgd", p, v.abs())
    tol = (2.2 * ds + 2.0 ** -11 + 2.0 ** -16)[..., None] * terms + (small * most * 127 * 2.0 ** -25)[..., None]
    tol = tol + 1.01 * HALF[q.dtype] * out.abs() + (2.0 ** -24 if q.dtype == torch.float16 else 2.0 ** -133)
    flat = lambda x: x.flatten(1, 2)  # noqa: E731
    return flat(out), flat(lse), flat(p), flat(tol), flat(1.1 * ds + 2.0 ** -18 * lse.abs().nan_to_num(0, 0, 0) + 1e-5), flat(ds)


def check(out, lse, want, what=""):
    o, ls, _, tol, ltol, _ = want
    assert torch.isfinite(out).all(), what
    off = (out.double() - o).abs() / tol
    assert (off <= 1).all(), f"{what}: {float(off.max())} of the bound at {(off == off.max()).nonzero()[0].tolist()}"
    if lse is not None:
        empty = torch.isinf(ls)
        assert (lse[empty] == -math.inf).all(), what
        assert ((lse.double() - ls)[~empty].abs() <= ltol[~empty]).all(), what


def masses(want, heads):
    """What the rows add to the mass of every token [L, H], and its bound: every weight's own error (its score's,
    lse's and the exponential's, 2^-18 together with the roundings of the sums)."""
    _, lse, p, _, ltol, ds = want
    R, Hq, L = p.shape
    p = p.view(R, heads, Hq // heads, L)
    rel = (2.2 * ds + 1.1 * ltol + 2.0 ** -18).view(R, heads, Hq // heads, 1)
    return p.sum((0, 2)).T, (p * rel).sum((0, 2)).T + 2.0 ** -100


def kept(mass, budget, first, last):
    """mass [L] (NaN, and -inf for tokens in no page, below everything) -> the positions that stay."""
    n = len(mass)
    if n <= budget:
        return list(range(n))
    key = [-math.inf if math.isnan(x) else x for x in mass]
    always = set(range(first)) | set(range(n - last, n))
    rest = sorted((j for j in range(n) if j not in always), key=lambda j: (-key[j], j))
    return sorted(always | set(rest[:budget - len(always)]))
