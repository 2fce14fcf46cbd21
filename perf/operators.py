"""Cases that measure the 4-bit key/value cache: writing it, reading it back, attention
over it (single tokens and prompts) and attention over the pages that a score selects.

The cache.  Page pool [page][kv head][block of 16 tokens][bytes], a block being

    K codes [16][D/2] | V codes [16][D/2] | K params [16][D/G][2] | V params [16][D/G][2]

with the params (s, c) of each group of G channels in the cache's type; a stored value
is x = c + s (u - 8), u in 0..15.  Where a channel's code sits in a row, and which row of
a block a token's V codes take, is given by ``_places``.  Beside the pool, bounds
[page][kv head][max, min][D] hold the extremes of each page's stored keys.

Sequences are batches of rows: sequence b has lens[b] tokens in the cache, its page j is
table[b][j], and its new rows (queries, or keys and values being written) are the last
starts[b + 1] - starts[b] of them."""
import math

import numpy as np
import torch

own = False  # True: the framework's operators; False: their plain form

_T = {"bf16": torch.bfloat16, "f16": torch.float16}


# ------------------------------------------------------------------------------- cases

def _case(name, op, batch, new, length, q_heads=0, kv_heads=8, dim=128, group=64, page=64, dtype="bf16", budget=0,
          ragged=False):
    return {"name": name, "op": op, "batch": batch, "new": new, "length": length, "q_heads": q_heads,
            "kv_heads": kv_heads, "dim": dim, "group": group, "page": page, "dtype": dtype, "budget": budget,
            "ragged": ragged}


def listed():
    """new: rows per sequence (the most of them where ragged); length: tokens per sequence
    with the new ones (where ragged, the longest; the others are spread below it)."""
    return [
        # one decode step of one user, the smallest write there is: latency
        _case("write_step_1", "write", 1, 1, 1021),
        # one decode step of a full server
        _case("write_step_256", "write", 256, 1, 2048, ragged=True),
        # one 8,192-token chunk of a long prompt
        _case("write_chunk_8192", "write", 1, 8192, 24576, dtype="f16"),
        # a few short prompts' caches taken out of the pool, odd lengths, small heads
        _case("read_prompts", "read", 5, 1999, 1999, kv_heads=3, dim=64, group=32, page=16, dtype="f16", ragged=True),
        # a 128K-token context read back whole (moved to another machine, or re-laid)
        _case("read_128k", "read", 1, 131072, 131072),
        # one user's next token after a short chat: latency
        _case("decode_1x777", "attention", 1, 1, 777, q_heads=32),
        # a server's decode step: 64 users, ragged contexts
        _case("decode_64x8k", "attention", 64, 1, 8191, q_heads=32, ragged=True),
        # two users of a 128K context, many heads to a key head, finer groups
        _case("decode_2x128k", "attention", 2, 1, 131072, q_heads=64, group=32, dtype="f16"),
        # short prompts of several users in one batch, a key head to every query head
        _case("prompt_ragged", "attention", 3, 333, 2500, q_heads=12, kv_heads=12, dim=64, group=32, page=32,
              dtype="f16", ragged=True),
        # one 8,192-token chunk of a prompt, the second of its kind
        _case("prompt_chunk_8192", "attention", 1, 8192, 16384, q_heads=32),
        # one user's next token over 16 pages of a 6K context
        _case("sparse_1x6k", "sparse", 1, 1, 6001, q_heads=32, budget=16),
        # 16 users of contexts up to 128K, each token over 64 pages
        _case("sparse_16x128k", "sparse", 16, 1, 131072, q_heads=64, budget=64, ragged=True),
    ]


def draw(rng):
    """Sizes over the listed cases' range: from one token of one user to the 128K contexts."""
    def size(lo, hi):
        return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))

    op = rng.choice(["write", "read", "attention", "attention", "sparse"])
    dim = rng.choice([64, 128, 128])
    kv = rng.choice([1, 2, 3, 4, 8, 8])
    c = _case("", op, 1, 1, 1, kv_heads=kv, dim=dim, group=rng.choice([32, 64] if dim == 64 else [32, 64, 64, 128]),
              page=rng.choice([16, 32, 64, 64, 128]), dtype=rng.choice(["bf16", "f16"]), ragged=rng.random() < 0.6)
    del c["name"]
    most = 1 << 18  # tokens of all sequences
    if op == "write":
        c["new"] = rng.choice([1, 1, size(2, 8192)])
        c["batch"] = size(1, 256 if c["new"] == 1 else max(1, 16384 // c["new"]))
        c["length"] = c["new"] + size(1, max(1, min(16384, most // c["batch"])))
    elif op == "read":
        c["batch"] = size(1, 32)
        c["new"] = c["length"] = size(1, min(131072, most // c["batch"]))
    else:
        c["q_heads"] = kv * rng.choice([1, 2, 4, 4, 7, 8])
        if op == "attention" and rng.random() < 0.5:  # prompts
            c["new"] = size(9, 4096)
            c["batch"] = size(1, max(1, min(8, 4096 // c["new"])))
            c["length"] = c["new"] + size(1, 4 * c["new"])
        else:
            c["new"] = rng.choice([1, 1, 1, 2, 4])
            c["batch"] = size(1, 64)
            c["length"] = c["new"] + size(1, min(131072, most // c["batch"]))
    if op == "sparse":
        c["budget"] = size(4, 64)
    return c


# ----------------------------------------------------------------------- the cache's form

def _places(dim, group, device):
    """For channel d: (byte in a K row, byte of a V row's piece order, shift of the nibble in
    that byte), and for token t of a block: (row of its V codes, xor of its V pieces).  Eight
    channels 0..7 of a 32-bit word take the nibbles 0 4 1 5 2 6 3 7."""
    d = torch.arange(dim, device=device)
    g, r = d // group, d % group
    quarter, rest = r // (group // 4), r % (group // 4)         # K: a quarter of every group side by side
    kn = quarter * (dim // 4) + g * (group // 4) + rest
    eighth, rest = r // (group // 8), r % (group // 8)          # V: an eighth (a "piece") of every group
    vn = eighth * (dim // 8) + g * (group // 8) + rest

    def nibble(n):
        at = (n % 8) // 2 + 4 * (n % 2)
        return (n // 8) * 4 + at // 2, (at % 2) * 4

    kb, ks = nibble(kn)
    vb, vs = nibble(vn)
    t = torch.arange(16, device=device)
    return {"kb": kb, "ks": ks, "vb": vb, "vs": vs, "vrow": (t & 8) | ((t & 1) << 2) | ((t >> 1) & 3),
            "vflip": ((t >> 2) & 1) * (dim // 4)}  # the byte offset of half a row's pieces


def _block_bytes(c):
    return 16 * (c["dim"] + 8 * (c["dim"] // c["group"]))


def _quantise(x, group, dtype):
    """x [..., D] fp32 -> codes [..., D] (uint8), params [..., D/G, 2] in the cache's type."""
    x = x.unflatten(-1, (-1, group))
    lo, hi = x.amin(-1), x.amax(-1)
    s = (hi / 15 - lo / 15).to(dtype)
    c = (lo + 8 * s.float()).to(dtype)
    fine = torch.isfinite(lo) & torch.isfinite(hi)
    s = torch.where(fine, s, torch.zeros_like(s))
    c = torch.where(fine, c, torch.full_like(c, math.nan))
    sf = s.float()[..., None]
    u = torch.clamp(torch.round((x - c.float()[..., None]) / sf) + 8, 0, 15)
    u = torch.where(sf > 0, u, torch.full_like(u, 8))
    return u.to(torch.uint8).flatten(-2), torch.stack((s, c), -1)


def _values(u, params, group):
    """The stored values in fp32: u [..., D], params [..., D/G, 2]."""
    s, c = params[..., 0].float()[..., None], params[..., 1].float()[..., None]
    return (c + s * (u.unflatten(-1, (-1, group)).float() - 8)).flatten(-2)


def _parts(pool, c):
    """Views of a pool [..., P/16, block bytes]: K codes, V codes, K params, V params by row."""
    d, n = c["dim"], c["dim"] // c["group"]
    rows = lambda lo, width: pool[..., lo:lo + 16 * width].unflatten(-1, (16, width))  # noqa: E731
    return rows(0, d // 2), rows(8 * d, d // 2), rows(16 * d, 4 * n), rows(16 * d + 64 * n, 4 * n)


def _pack(u, byte, shift):
    """codes [..., D] -> bytes [..., D/2]: channel d's nibble at (byte, shift)."""
    out = torch.zeros(u.shape[:-1] + (u.shape[-1] // 2,), dtype=torch.int32, device=u.device)
    return out.index_add_(out.dim() - 1, byte, u.int() << shift.int()).to(torch.uint8)


def _write(c, pool, at, page, offset, k, v):
    """Quantise k, v [N, H, D] into rows (page [N], offset [N]) of the pool."""
    dtype, heads = _T[c["dtype"]], torch.arange(c["kv_heads"], device=pool.device)
    kc, vc, kp, vp = _parts(pool, c)
    blk, row = (offset // 16)[:, None], (offset % 16)[:, None]
    pg, hd = page[:, None], heads[None, :]
    u, p = _quantise(k.float(), c["group"], dtype)
    kc[pg, hd, blk, row] = _pack(u, at["kb"], at["ks"])
    kp[pg, hd, blk, row] = p.flatten(-2).view(torch.uint8)
    u, p = _quantise(v.float(), c["group"], dtype)
    bytes_ = _pack(u, at["vb"], at["vs"])
    order = torch.arange(c["dim"] // 2, device=pool.device)[None, :] ^ at["vflip"][offset % 16][:, None]
    bytes_ = bytes_.gather(-1, order[:, None, :].expand_as(bytes_))
    vc[pg, hd, blk, at["vrow"][row]] = bytes_
    vp[pg, hd, blk, row] = p.flatten(-2).view(torch.uint8)


def _unpack(c, at, pool):
    """Blocks of a pool [..., P/16, block bytes] -> K, V [..., P, D] in fp32."""
    dtype = _T[c["dtype"]]
    kc, vc, kp, vp = _parts(pool, c)
    params = lambda p: p.contiguous().view(dtype).unflatten(-1, (-1, 2))  # noqa: E731
    ku = (kc[..., at["kb"]] >> at["ks"].to(torch.uint8)) & 15
    row = at["vrow"][:, None]
    vu = (vc[..., row, at["vb"][None, :] ^ at["vflip"][:, None]] >> at["vs"].to(torch.uint8)) & 15
    return (_values(ku, params(kp), c["group"]).flatten(-3, -2), _values(vu, params(vp), c["group"]).flatten(-3, -2))


# ------------------------------------------------------------------------------- inputs

def _lengths(c):
    """Tokens and new rows of each sequence, the same for every seed; the first sequence has
    the most of both."""
    r = np.random.RandomState((c["batch"] * 1000003 + c["length"] * 101 + c["new"]) % (1 << 31))
    b, new, length = c["batch"], c["new"], c["length"]
    n = np.full(b, new)
    if c["ragged"] and new > 8:
        n[1:] = r.randint(max(1, new // 3), new + 1, b - 1)
    total = np.full(b, length)
    if c["ragged"]:
        total[1:] = np.maximum(n[1:], r.randint(max(1, length // 4), length + 1, b - 1))
    return (n.copy() if c["op"] == "read" else total), n


def prepare(case, seed):
    c = dict(case)
    dev, dtype = torch.device("cuda"), _T[c["dtype"]]
    lens, new = _lengths(c)
    gen = torch.Generator(device=dev)
    gen.manual_seed(int(seed))
    b, page, heads, dim = c["batch"], c["page"], c["kv_heads"], c["dim"]
    pages = -(-lens // page)
    cols, count = int(pages.max()), int(pages.sum())
    spare = 7  # pages of nobody
    ids = torch.randperm(count + spare, generator=gen, device=dev).int()
    table = torch.full((b, cols), -1, dtype=torch.int32, device=dev)
    for i, first in enumerate(np.cumsum(pages) - pages):
        table[i, :pages[i]] = ids[first:first + pages[i]]
    at = _places(dim, c["group"], dev)
    pool = torch.zeros(count + spare, heads, page // 16, _block_bytes(c), dtype=torch.uint8, device=dev)
    bounds = torch.zeros(count + spare, heads, 2, dim, dtype=dtype, device=dev)
    # keys have channels of their own size and offset, values are plain
    size = torch.exp(0.5 * torch.randn(heads, dim, generator=gen, device=dev))
    mean = 0.5 * torch.randn(heads, dim, generator=gen, device=dev)

    def rows(n):
        k = torch.randn(n, heads, dim, generator=gen, device=dev) * size + mean
        return k.to(dtype), torch.randn(n, heads, dim, generator=gen, device=dev).to(dtype)

    held = lens - new if c["op"] == "write" else lens
    for i in range(b):  # the tokens that are in the cache before the call
        for first in range(0, int(held[i]), 16384):
            pos = torch.arange(first, min(first + 16384, int(held[i])), device=dev)
            _write(c, pool, at, table[i, pos // page].long(), pos % page, *rows(len(pos)))
    starts = np.concatenate([[0], np.cumsum(new)])
    st = {"case": c, "pool": pool, "bounds": bounds, "table": table, "at": at, "max_new": int(new.max()),
          "lens": torch.from_numpy(lens).int().to(dev), "starts": torch.from_numpy(starts).int().to(dev),
          "uniform": bool((new == new[0]).all()), "rows": int(starts[-1]), "scale": 1 / math.sqrt(dim)}
    if c["op"] in ("write", "sparse"):  # the bounds of the tokens that are in the cache
        have = torch.from_numpy(held).to(dev)
        for i in range(b):
            n = -(-int(held[i]) // page)
            for first in range(0, n, 256):
                j = torch.arange(first, min(first + 256, n), device=dev)
                bounds[table[i, j].long()] = _page_bounds(st, table[i, j].long(), j, have[i].expand(len(j)))
    if c["op"] == "write":
        st["k"], st["v"] = rows(st["rows"])
    elif c["op"] == "read":
        st["k"], st["v"] = (torch.empty(st["rows"], heads, dim, dtype=dtype, device=dev) for _ in range(2))
    else:
        # queries lean on their key head's channels, so that scores are not all alike
        q = torch.randn(st["rows"], heads, c["q_heads"] // heads, dim, generator=gen, device=dev)
        q = q + 0.5 * torch.randn(st["rows"], heads, 1, dim, generator=gen, device=dev)
        st["q"] = q.flatten(1, 2).to(dtype)
    return st


# --------------------------------------------------------------------------- plain forms

def _page_bounds(st, page_ids, index, lens):
    """[n, H, 2, D]: extremes of the stored keys of pages `page_ids`, each its sequence's
    page `index` of a sequence of `lens` tokens."""
    c = st["case"]
    k, _ = _unpack(c, st["at"], st["pool"][page_ids])
    inside = index[:, None] * c["page"] + torch.arange(c["page"], device=k.device) < lens[:, None]
    inside = inside[:, None, :, None]
    hi = torch.where(inside, k, torch.full_like(k, -math.inf)).amax(2)
    lo = torch.where(inside, k, torch.full_like(k, math.inf)).amin(2)
    return torch.stack((hi, lo), 2).to(_T[c["dtype"]])


def _positions(st):
    """Sequence and position of every new row."""
    starts = st["starts"].long()
    i = torch.arange(st["rows"], device=starts.device)
    seq = torch.bucketize(i, starts[1:], right=True)
    return seq, st["lens"].long()[seq] - starts[seq + 1] + i


def _rows_of(st, seq, pos):
    """K, V [N, H, D] of (sequence, position) pairs."""
    c = st["case"]
    page, off = st["table"].long()[seq, pos // c["page"]], pos % c["page"]
    k, v = _unpack(c, st["at"], st["pool"][page, :, off // 16][:, :, None])
    pick = (off % 16)[:, None, None, None].expand(-1, k.shape[1], 1, k.shape[3])
    return k.gather(2, pick)[:, :, 0], v.gather(2, pick)[:, :, 0]


def _plain_write(st):
    c = st["case"]
    seq, pos = _positions(st)
    _write(c, st["pool"], st["at"], st["table"].long()[seq, pos // c["page"]], pos % c["page"], st["k"], st["v"])
    # the pages that the new rows touch (a page named twice gets the same bounds twice)
    lens = st["lens"].long()
    first = (lens - (st["starts"][1:] - st["starts"][:-1]).long()) // c["page"]
    most = (st["max_new"] + c["page"] - 2) // c["page"] + 1
    j = torch.minimum(first[:, None] + torch.arange(most, device=lens.device), (lens[:, None] - 1) // c["page"])
    ids = st["table"].long().gather(1, j).flatten()
    new = _page_bounds(st, ids, j.flatten(), lens[:, None].expand_as(j).flatten())
    st["bounds"][ids] = new
    k, v = _rows_of(st, seq, pos)
    return {"k": k.to(st["k"].dtype), "v": v.to(st["v"].dtype), "bounds": st["bounds"]}


def _plain_read(st):
    k, v = _rows_of(st, *_positions(st))
    return {"k": k.to(st["k"].dtype), "v": v.to(st["v"].dtype)}


def _softmax_rows(s, seen):
    s = torch.where(seen, s, torch.full_like(s, -math.inf))
    top = s.amax(-1, keepdim=True)
    p = torch.exp(s - torch.where(torch.isfinite(top), top, torch.zeros_like(top)))
    total = p.sum(-1, keepdim=True)
    return p / torch.where(total > 0, total, torch.ones_like(total))


def _plain_attention(st):
    c, n = st["case"], st["max_new"]
    dev, heads = st["q"].device, c["kv_heads"]
    k, v = _unpack(c, st["at"], st["pool"][st["table"].long().clamp_min(0)].transpose(1, 2))  # [B, H, pages, P, D]
    k, v = k.flatten(2, 3), v.flatten(2, 3)
    starts, lens = st["starts"].long(), st["lens"].long()
    j = torch.arange(n, device=dev)
    i = (starts[:-1, None] + j).clamp_max(st["rows"] - 1)                       # [B, n]: every sequence padded to n rows
    last = lens[:, None] - (starts[1:] - starts[:-1])[:, None] + j              # position of each row
    q = st["q"].float()[i].unflatten(2, (heads, -1)).permute(0, 2, 1, 3, 4)     # [B, H, n, g, D]
    shape = q.shape
    s = q.flatten(2, 3) @ k.transpose(-1, -2) * st["scale"]
    seen = torch.arange(k.shape[2], device=dev) <= torch.minimum(last, lens[:, None] - 1)[:, :, None]
    seen = seen[:, None, :, None, :].expand(-1, 1, -1, shape[3], -1).flatten(2, 3)
    o = (_softmax_rows(s, seen) @ v).view(shape).permute(0, 2, 1, 3, 4).flatten(2, 3)
    seq, _ = _positions(st)
    return {"out": o[seq, torch.arange(st["rows"], device=dev) - starts[seq]].to(st["q"].dtype)}


def _tree_sum(x):
    """Sum over the last axis (a power of two) by adjacent pairs, level by level."""
    return x[..., 0] if x.shape[-1] == 1 else _tree_sum(x[..., 0::2] + x[..., 1::2])


def _head_sum(q):
    """Sum over axis 2, ascending, one addition after the other."""
    return q[:, :, 0] if q.shape[2] == 1 else _head_sum(torch.cat((q[:, :, :1] + q[:, :, 1:2], q[:, :, 2:]), 2))


def _plain_select(st):
    """[N, H, budget]: the first page, the last page, and the pages of the highest scores."""
    c = st["case"]
    seq, pos = _positions(st)
    table = st["table"].long().clamp_min(0)
    q = _head_sum(st["q"].float().unflatten(1, (c["kv_heads"], -1)))            # [N, H, D]
    ext = st["bounds"][table].transpose(1, 2).float()                           # [B, H, pages, 2, D]
    prod = q[:, :, None, None] * ext[seq]
    score = _tree_sum(torch.maximum(prod[:, :, :, 0], prod[:, :, :, 1]))
    score = torch.where(torch.isnan(score), torch.full_like(score, -math.inf), score)
    j = torch.arange(table.shape[1], device=table.device)
    seen = (pos // c["page"])[:, None, None]
    rank = torch.where((j == 0) | (j == seen), 2.0, 1.0).expand_as(score)       # always, by score, never
    rank = torch.where(j <= seen, rank, torch.zeros_like(rank))
    by_score = torch.sort(score, dim=-1, descending=True, stable=True).indices
    order = torch.sort(rank.gather(-1, by_score), dim=-1, descending=True, stable=True).indices
    pick = by_score.gather(-1, order)[..., :c["budget"]]
    none = torch.full_like(pick, 1 << 30)
    pick = torch.sort(torch.where(pick <= seen, pick, none), -1).values
    short = torch.full(pick.shape[:2] + (c["budget"] - pick.shape[2],), 1 << 30, device=pick.device)
    pick = torch.cat((pick, short), -1)
    return torch.where(pick < (1 << 30), pick, torch.full_like(pick, -1)).int()


def _plain_sparse(st):
    c = st["case"]
    pick = _plain_select(st)
    seq, pos = _positions(st)
    at = pick.long().clamp_min(0)
    ids = st["table"].long()[seq[:, None, None], at]
    heads = torch.arange(c["kv_heads"], device=ids.device)[None, :, None]
    k, v = _unpack(c, st["at"], st["pool"][ids, heads])                         # [N, H, budget, P, D]
    where = at[..., None] * c["page"] + torch.arange(c["page"], device=ids.device)
    seen = ((pick >= 0)[..., None] & (where <= pos[:, None, None, None])).flatten(2)[:, :, None]
    q = st["q"].float().unflatten(1, (c["kv_heads"], -1))
    p = _softmax_rows(q @ k.flatten(2, 3).transpose(-1, -2) * st["scale"], seen)
    return {"pages": pick, "out": (p @ v.flatten(2, 3)).flatten(1, 2).to(st["q"].dtype)}


_PLAIN = {"write": _plain_write, "read": _plain_read, "attention": _plain_attention, "sparse": _plain_sparse}


def run(state):
    c = state["case"]
    if not own:
        return _PLAIN[c["op"]](state)
    cache = state.get("cache")
    if cache is None:  # the handle that a program makes once
        from moe_expert_layer_sorted_gb300 import KVCache
        cache = state["cache"] = KVCache(state["pool"], page_size=c["page"], head_dim=c["dim"], group_size=c["group"],
                                         dtype=_T[c["dtype"]], bounds=state["bounds"])
    batch = dict(table=state["table"], lens=state["lens"])
    if state["uniform"]:
        shape = (c["batch"], state["max_new"])
    else:
        shape = (state["rows"],)
        batch.update(starts=state["starts"], max_new=state["max_new"])
    if c["op"] in ("write", "read"):
        if c["op"] == "write":
            cache.append(state["k"].view(*shape, *state["k"].shape[1:]), state["v"].view(*shape, *state["v"].shape[1:]),
                         **batch)
        k, v = torch.empty_like(state["k"]), torch.empty_like(state["v"])
        cache.read(k.view(*shape, *k.shape[1:]), v.view(*shape, *v.shape[1:]), **batch)
        return {"k": k, "v": v, "bounds": state["bounds"]} if c["op"] == "write" else {"k": k, "v": v}
    q = state["q"].view(*shape, *state["q"].shape[1:])
    out = torch.empty_like(state["q"])
    if c["op"] == "attention":
        cache.attention(q, out.view(q.shape), scale=state["scale"], **batch)
        return {"out": out}
    pages = torch.empty(state["rows"], c["kv_heads"], c["budget"], dtype=torch.int32, device=out.device)
    cache.select(q, pages, **batch)
    cache.attention(q, out.view(q.shape), scale=state["scale"], pages=pages, **batch)
    return {"pages": pages, "out": out}


def work(case):
    """Every input once, every output once; a stored row and head takes D + 8 D/G bytes."""
    c = case
    lens, new = (x.astype(np.float64) for x in _lengths(c))
    row = c["kv_heads"] * (c["dim"] + 8 * (c["dim"] // c["group"]))
    wide = 4.0 * c["kv_heads"] * c["dim"]                # a row's keys and values in 16 bits
    qo = 4.0 * c["q_heads"] * c["dim"]                   # a row's queries and outputs
    ends = c["kv_heads"] * 4.0 * c["dim"]                # a page's bounds
    n = float(new.sum())
    if c["op"] == "read":
        return {"bytes": n * (row + wide), "flops": 2.0 * n * wide}
    if c["op"] == "write":                               # written, and read back
        touched = float(((lens - 1) // c["page"] - (lens - new) // c["page"] + 1).sum())
        return {"bytes": n * (2 * wide + 2 * row) + 2 * touched * ends, "flops": 5.0 * n * wide}
    seen = new * lens - new * (new - 1) / 2              # visible (row, token) pairs of a sequence
    if c["op"] == "attention":
        return {"bytes": float(lens.sum()) * row + n * qo, "flops": 4.0 * c["q_heads"] * c["dim"] * float(seen.sum())}
    pages = -(-lens // c["page"])
    read = np.minimum(pages, c["budget"]) * c["page"] * new
    return {"bytes": float((pages * ends).sum()) + float(np.minimum(read, lens * new).sum()) * row + n * qo
            + 4.0 * n * c["kv_heads"] * c["budget"],
            "flops": float((pages * new).sum()) * 4 * c["kv_heads"] * c["dim"] + 4.0 * c["q_heads"] * c["dim"] * float(read.sum())}


# ------------------------------------------------------------- the definition in 64 bits

def exact(case, seed):
    """Row by row from the definition: the groups' own arithmetic, and attention as it is
    written down, in 64 bits; the choice of pages is a whole-number output and has none."""
    st = prepare(case, seed)
    c, dtype = st["case"], _T[case["dtype"]]
    dev, heads, dim, group, page = st["pool"].device, c["kv_heads"], c["dim"], c["group"], c["page"]
    lens, starts = st["lens"].tolist(), st["starts"].tolist()

    def stored(x):
        """What becomes of 16-bit rows [n, H, D] in the cache."""
        g = x.double().reshape(*x.shape[:-1], dim // group, group)
        lo = g.min(-1, keepdim=True).values
        s = ((g.max(-1, keepdim=True).values - lo) / 15).to(dtype).double()
        mid = (lo + 8 * s).to(dtype).double()
        u = ((g - mid) / torch.where(s > 0, s, torch.ones_like(s))).round().clamp(-8, 7) * (s > 0)
        return (mid + s * u).reshape(x.shape)

    def bits(n):  # where the nibble of the n-th channel of a row's order starts
        return (n // 8) * 32 + ((n % 8) // 2 + 4 * (n % 2)) * 4

    d = np.arange(dim)
    kbit = bits((d % group) // (group // 4) * (dim // 4) + d // group * (group // 4) + d % (group // 4))
    vbit = bits((d % group) // (group // 8) * (dim // 8) + d // group * (group // 8) + d % (group // 8))
    kbit, vbit = torch.from_numpy(kbit).to(dev), torch.from_numpy(vbit).to(dev)

    def held(b, h, first, last):
        """K, V [last - first, D] of tokens first..last-1 of sequence b's head h."""
        pos = torch.arange(first, last, device=dev)
        off = pos % page
        block = st["pool"][st["table"][b].long()[pos // page], h, off // 16]    # [n, bytes]
        r, n = off % 16, dim // group
        vr = (r // 8) * 8 + (r % 2) * 4 + (r // 2) % 4
        flip = (r // 4) % 2 * (dim // 4)

        def side(base, row, bit, xor, params):
            byte = base + row[:, None] * (dim // 2) + ((bit // 8)[None, :] ^ xor[:, None])
            u = (block.gather(1, byte).long() >> (bit % 8)[None, :]) % 16 - 8
            where = params + (r * 4 * n)[:, None] + torch.arange(4 * n, device=dev)
            sc = block.gather(1, where).view(dtype).double().reshape(-1, n, 2)
            return (sc[:, :, 1, None] + sc[:, :, 0, None] * u.double().reshape(-1, n, group)).reshape(-1, dim)

        return side(0, r, kbit, 0 * r, 16 * dim), side(8 * dim, vr, vbit, flip, 16 * dim + 64 * n)

    if c["op"] == "read":
        k, v = (torch.empty(st["rows"], heads, dim, dtype=torch.float64, device=dev) for _ in range(2))
        for b in range(c["batch"]):
            for h in range(heads):
                k[starts[b]:starts[b + 1], h], v[starts[b]:starts[b + 1], h] = held(b, h, lens[b] - (starts[b + 1] - starts[b]), lens[b])
        return {"k": k, "v": v}
    if c["op"] == "write":
        k, v, ends = stored(st["k"]), stored(st["v"]), st["bounds"].double()
        for b in range(c["batch"]):
            first = lens[b] - (starts[b + 1] - starts[b])
            for j in range(first // page, (lens[b] - 1) // page + 1):
                a, z = max(first, j * page), min(lens[b], (j + 1) * page)
                rows = k[starts[b] + a - first:starts[b] + z - first].to(dtype).double()
                hi, lo, e = rows.max(0).values, rows.min(0).values, ends[int(st["table"][b, j])]
                if a > j * page:  # the page held tokens before
                    hi, lo = torch.maximum(hi, e[:, 0]), torch.minimum(lo, e[:, 1])
                e[:, 0], e[:, 1] = hi, lo
        return {"k": k, "v": v, "bounds": ends}
    per = c["q_heads"] // heads
    out = torch.zeros(st["rows"], c["q_heads"], dim, dtype=torch.float64, device=dev)
    if c["op"] == "sparse":
        pick = _plain_select(st).tolist()
    for b in range(c["batch"]):
        n = starts[b + 1] - starts[b]
        for h in range(heads):
            k, v = held(b, h, 0, lens[b])
            for a in range(0, n, 1024):
                z = min(n, a + 1024)
                q = st["q"][starts[b] + a:starts[b] + z, h * per:(h + 1) * per].double()
                s = torch.einsum("ngd,ld->ngl", q, k) / math.sqrt(dim)
                pos = torch.arange(lens[b], device=dev)
                hidden = pos[None, :] > lens[b] - n + torch.arange(a, z, device=dev)[:, None]
                if c["op"] == "sparse":
                    for i in range(a, z):
                        hidden[i - a] |= ~torch.isin(pos // page, torch.tensor(pick[starts[b] + i][h], device=dev))
                w = torch.softmax(s.masked_fill(hidden[:, None], -math.inf), -1)
                out[starts[b] + a:starts[b] + z, h * per:(h + 1) * per] = torch.einsum("ngl,ld->ngd", w, v)
    return {"pages": None, "out": out} if c["op"] == "sparse" else {"out": out}
