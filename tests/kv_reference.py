"""Plain implementation of the 4-bit key/value cache for the tests: the format from its
definition, attention in 64 bits, page selection with the documented summation order."""
import math

import numpy as np
import torch

UNIT = {torch.bfloat16: 2.0 ** -9, torch.float16: 2.0 ** -12}  # half a unit in the last place, relative


def quantise(x, group):
    """16-bit x [..., D] -> (codes u [..., D] uint8, s, c [..., D/G]) by the definition, in fp32."""
    g = x.float().unflatten(-1, (-1, group))
    lo, hi = g.amin(-1), g.amax(-1)
    s = (hi / 15 - lo / 15).to(x.dtype)
    c = (lo.double() + 8 * s.double()).float().to(x.dtype)  # one fp32 rounding: 8 s alone may overflow
    bad = ~torch.isfinite(g).all(-1)
    s[bad], c[bad] = 0.0, math.nan
    u = ((g - c.float()[..., None]) / s.float()[..., None]).round().add(8).clamp(0, 15)
    u = torch.where(s.float()[..., None] > 0, u, torch.full_like(u, 8))
    return u.to(torch.uint8).flatten(-2), s, c


def values(x, group):
    """The stored values of x in 64 bits."""
    u, s, c = quantise(x, group)
    return (c.double()[..., None] + s.double()[..., None] * (u.unflatten(-1, (-1, group)).double() - 8)).flatten(-2)


def decode_block(block, D, G, dtype):
    """One block's bytes (numpy uint8) -> K codes, V codes [16][D], K params, V params [16][D/G][2]."""
    n = D // G
    kc, vc = block[:8 * D].reshape(16, D // 2), block[8 * D:16 * D].reshape(16, D // 2)
    par = torch.from_numpy(block[16 * D:].copy()).view(dtype).reshape(2, 16, n, 2)
    ku, vu = np.zeros((16, D), np.uint8), np.zeros((16, D), np.uint8)

    def nibble(row, i):  # the i-th channel of a row's order
        word, e = divmod(i, 8)
        at = e // 2 + 4 * (e % 2)
        return (row[word * 4 + at // 2] >> (4 * (at % 2))) & 15

    for t in range(16):
        row = (t & 8) | ((t & 1) << 2) | ((t >> 1) & 3)
        v = vc[row]
        if t & 4:
            v = np.concatenate([v[D // 4:], v[:D // 4]])
        for d in range(D):
            g, r = divmod(d, G)
            ku[t, d] = nibble(kc[t], r // (G // 4) * (D // 4) + g * (G // 4) + r % (G // 4))
            vu[t, d] = nibble(v, r // (G // 8) * (D // 8) + g * (G // 8) + r % (G // 8))
    return ku, vu, par[0], par[1]


def attention(q, k, v, seen, scale):
    """q [R, Hq, D], k, v [L, H, D] (64 bits), seen [R, L] or [R, H, L] bool -> out, lse, the
    a-priori bounds of both for a kernel that rounds k, the probabilities and the output to
    q's type and sums in fp32."""
    u = UNIT[q.dtype]
    R, Hq, D = q.shape
    L, H, _ = k.shape
    qd = q.double().view(R, H, Hq // H, D)
    if seen.dim() == 2:
        seen = seen[:, None].expand(R, H, L)
    if L == 0:
        z = torch.zeros(R, Hq, D, dtype=torch.float64, device=q.device)
        return z, torch.full((R, Hq), -math.inf, dtype=torch.float64, device=q.device), z, z[..., 0]
    k0, v0 = (torch.where(seen.any(0).T[:, :, None], x, torch.zeros_like(x)) for x in (k, v))  # unseen may be anything
    s = torch.einsum("rhgd,lhd->rhgl", qd, k0) * scale
    mag = torch.einsum("rhgd,lhd->rhgl", qd.abs(), k0.abs()) * abs(scale)
    s = s.masked_fill(~seen[:, :, None], -math.inf)
    top = s.amax(-1, keepdim=True)
    p = torch.exp(s - torch.where(torch.isfinite(top), top, torch.zeros_like(top)))
    tot = p.sum(-1, keepdim=True)
    out = torch.einsum("rhgl,lhd->rhgd", p / tot.clamp_min(1e-300), v0)
    lse = torch.where(tot[..., 0] > 0, top[..., 0] + torch.log(tot[..., 0].clamp_min(1e-300)), top[..., 0])
    # errors: a score by (u + 2^-16) of its terms' magnitude (k rounded, fp32 sums of up to
    # 2^7 terms), so every weight by twice the largest; weights and output rounded once each
    ds = torch.where(seen[:, :, None], mag, torch.zeros_like(mag)).amax(-1) * (u + 2.0 ** -16) + 2.0 ** -16
    vmax = torch.where(seen.any(0).T[:, :, None], v0.abs(), torch.zeros_like(v0)).amax((0, 2))[None, :, None]
    tol = (2.2 * ds + 1.1 * u + 2.0 ** -14) * vmax
    tol = tol[..., None] + 1.1 * u * out.abs() + 2.0 ** -24
    return out.flatten(1, 2), lse.flatten(1, 2), tol.flatten(1, 2), (1.1 * ds + 2.0 ** -18 * lse.abs().nan_to_num(0, 0, 0)).flatten(1, 2)


def scores(qs, hi, lo):
    """fp32 scores with the documented order: qs [D], hi, lo [pages, D] fp32."""
    x = torch.maximum(qs * hi, qs * lo)
    while x.shape[-1] > 1:
        x = x[..., 0::2] + x[..., 1::2]
    return x[..., 0]


def select(q, hi, lo, pages, budget, first, last):
    """q [g, D] 16-bit, hi, lo [pages, D] 16-bit: the list of `budget` entries."""
    if pages <= budget:
        return list(range(pages)) + [-1] * (budget - pages)
    qs = q[0].float()
    for h in range(1, q.shape[0]):
        qs = qs + q[h].float()
    sc = scores(qs, hi[:pages].float(), lo[:pages].float()).tolist()
    sc = [-math.inf if math.isnan(x) else x for x in sc]
    keep = set(range(first)) | set(range(pages - last, pages))
    rest = sorted((j for j in range(pages) if j not in keep), key=lambda j: (-sc[j], j))
    return sorted(list(keep) + rest[:budget - len(keep)])
