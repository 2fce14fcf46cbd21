"""Cases that measure the 8-bit key/value cache: writing it, attention over it (single tokens and
prompts), attention that also adds up the weight every token gets, and the eviction of the tokens
that got least.

The cache.  Page pool [page][kv head][block of 16 tokens][bytes], a block being

    K codes [16][D] | V codes [8 token pairs][D][2] | params: K step, V step (fp32), K marks, V marks (16 bits), 0

with codes u + 128, u in -127..127, and the stored value x = s u, s being the step that the block's
16 tokens share (keys and values apart); a token's mark says that its keys (values) held something
that was not finite: they read as NaN.  Within a row of K codes and a pair of V codes the pieces of
16 bytes change places, ``_places``.  A write of some tokens of a block whose first ones are there
already keeps the larger step of the two and turns the older codes to it where it grows.

Beside the pool, mass [page][kv head][page size] holds in fp32 what weight the softmax has given to
each token, summed over the rows and query heads that saw it.  An eviction keeps, of every head of a
sequence, the first and the last tokens and those of the largest mass, `budget` in all, and moves them
together in their order; a block of moved tokens takes the largest of their steps."""
import math

import numpy as np
import torch

own = False  # True: the framework's operators; False: their plain form

_T = {"bf16": torch.bfloat16, "f16": torch.float16}


# ------------------------------------------------------------------------------- cases

def _case(name, op, batch, new, length, q_heads=0, kv_heads=8, dim=128, page=64, dtype="bf16", budget=0, first=0, last=0,
          ragged=False):
    return {"name": name, "op": op, "batch": batch, "new": new, "length": length, "q_heads": q_heads,
            "kv_heads": kv_heads, "dim": dim, "page": page, "dtype": dtype, "budget": budget, "first": first, "last": last,
            "ragged": ragged}


def listed():
    """new: rows per sequence (the most of them where ragged); length: tokens per sequence with the
    new ones (where ragged, the longest; the others are spread below it)."""
    return [
        # one decode step of a full server: a row each, into blocks that hold tokens
        _case("write_step_256", "write", 256, 1, 2048, ragged=True),
        # one 8,192-token chunk of a long prompt, not at a block's start
        _case("write_chunk_8192", "write", 1, 8192, 24571, dtype="f16"),
        # one user's next token after a short chat: latency
        _case("decode_1x777", "attention", 1, 1, 777, q_heads=32),
        # a server's decode step: 64 users, ragged contexts
        _case("decode_64x8k", "attention", 64, 1, 8191, q_heads=32, ragged=True),
        # two users of a 128K context, many heads to a key head
        _case("decode_2x128k", "attention", 2, 1, 131072, q_heads=64, dtype="f16"),
        # short prompts of several users in one batch, a key head to every query head
        _case("prompt_ragged", "attention", 3, 333, 2500, q_heads=12, kv_heads=12, dim=64, page=32, dtype="f16", ragged=True),
        # one 8,192-token chunk of a prompt, the second of its kind
        _case("prompt_chunk_8192", "attention", 1, 8192, 16384, q_heads=32),
        # one user's next token, its weights counted: latency
        _case("weigh_1x2k", "weigh", 1, 1, 2047, q_heads=32),
        # 32 users' next tokens over caches that are kept at some 4K tokens each
        _case("weigh_32x4k", "weigh", 32, 1, 4160, q_heads=32, ragged=True),
        # a prompt that is longer than what will be kept of it
        _case("weigh_prompt_4096", "weigh", 1, 4096, 4096, q_heads=32, dtype="f16"),
        # 32 users' caches back to 4K tokens after some steps
        _case("evict_32x4k", "evict", 32, 0, 4608, budget=4096, first=4, last=256, ragged=True),
        # half of a 128K context
        _case("evict_1x128k", "evict", 1, 0, 131072, budget=65536, first=64, last=4096),
    ]


def draw(rng):
    """Sizes over the listed cases' range: from one token of one user to the 128K contexts."""
    def size(lo, hi):
        return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))

    op = rng.choice(["write", "attention", "attention", "weigh", "weigh", "evict"])
    kv = rng.choice([1, 2, 3, 4, 8, 8])
    c = _case("", op, 1, 1, 1, kv_heads=kv, dim=rng.choice([64, 128, 128]), page=rng.choice([16, 32, 64, 64, 128]),
              dtype=rng.choice(["bf16", "f16"]), ragged=rng.random() < 0.6)
    del c["name"]
    most = 1 << 18  # tokens of all sequences
    if op == "write":
        c["new"] = rng.choice([1, 1, size(2, 8192)])
        c["batch"] = size(1, 256 if c["new"] == 1 else max(1, 16384 // c["new"]))
        c["length"] = c["new"] + size(1, max(1, min(16384, most // c["batch"])))
    elif op == "evict":
        c["new"] = 0
        c["batch"] = size(1, 32)
        c["length"] = size(40, min(131072, most // c["batch"]))
        c["budget"] = size(8, c["length"])
        c["first"] = rng.choice([0, 1, min(4, c["budget"] // 4)])
        c["last"] = size(1, max(1, c["budget"] // 4))
    else:
        c["q_heads"] = kv * rng.choice([1, 2, 4, 4, 7, 8])
        if rng.random() < 0.5:  # prompts
            c["new"] = size(9, 4096)
            c["batch"] = size(1, max(1, min(8, 4096 // c["new"])))
            c["length"] = c["new"] + size(1, 2 * c["new"])
        else:
            c["new"] = rng.choice([1, 1, 1, 2, 4])
            c["batch"] = size(1, 64)
            c["length"] = c["new"] + size(1, min(131072, most // c["batch"]))
    return c


# ----------------------------------------------------------------------- the cache's form

def _places(dim, device):
    """Byte in a block of every token's every channel: keys, values [16, D]."""
    t, d = torch.arange(16, device=device)[:, None], torch.arange(dim, device=device)
    k = t * dim + ((d // 16) ^ ((t & 1) * (4 if dim == 128 else 0))) * 16 + d % 16
    p = (t // 2) % 4
    turn = (p & 1) | ((p >> 1) << 2) if dim == 128 else 2 * p
    v = 16 * dim + (t // 2) * 2 * dim + ((d // 8) ^ turn) * 16 + d % 8 * 2 + t % 2
    return {"k": k, "v": v}


def _block_bytes(c):
    return 32 * c["dim"] + 16


def _params(blocks, dim):
    """Steps [..., 2] in fp32 and marks [..., 2, 16] of blocks [..., bytes]."""
    p = blocks[..., 32 * dim:]
    bits = p[..., 8:12].unflatten(-1, (2, 2)).int()
    bits = bits[..., 0] | bits[..., 1] << 8
    return p[..., :8].contiguous().view(torch.float32), (bits[..., None] >> torch.arange(16, device=p.device)) & 1 > 0


def _codes(blocks, at):
    """u [..., 2, 16, D] of blocks [..., bytes]."""
    pick = torch.stack((at["k"], at["v"]))
    return blocks[..., pick.flatten()].unflatten(-1, pick.shape).int() - 128


def _blocks(u, s, marks, at):
    """Blocks [..., bytes] of codes u [..., 2, 16, D], steps s [..., 2], marks [..., 2, 16]."""
    dim = u.shape[-1]
    out = torch.zeros(u.shape[:-3] + (32 * dim + 16,), dtype=torch.uint8, device=u.device)
    out[..., torch.stack((at["k"], at["v"])).flatten()] = (u + 128).flatten(-3).to(torch.uint8)
    out[..., 32 * dim:32 * dim + 8] = s.contiguous().view(torch.uint8)
    bits = (marks.int() << torch.arange(16, device=u.device)).sum(-1)
    out[..., 32 * dim + 8:32 * dim + 12] = torch.stack((bits & 255, bits >> 8), -1).flatten(-2).to(torch.uint8)
    return out


def _whole(num, den):
    """num / den to the nearest whole number (0 where den is 0), in 64 bits: what is near a half is told apart."""
    den = den.double()
    return torch.where(den > 0, num / torch.where(den > 0, den, torch.ones_like(den)), torch.zeros_like(num)).round().int()


def _write(old, x, is_old, is_new, at):
    """Blocks old [..., bytes] with the tokens x [..., 2, 16, D] written where is_new [..., 16]; those
    where is_old were there before."""
    x = x.float()
    fine = torch.isfinite(x).all(-1) & is_new[..., None, :]
    top = torch.where(fine[..., None], x, torch.zeros_like(x)).abs().amax((-2, -1))
    s = (top.double() / 127).float()
    was, marks = _params(old, x.shape[-1])
    has = is_old.any(-1)[..., None]
    was = torch.where(has, was, torch.zeros_like(was))
    s = torch.maximum(s, was)
    u = _codes(old, at)
    turned = _whole(u.double() * was.double()[..., None, None], s[..., None, None].expand_as(u))
    u = torch.where((was < s)[..., None, None], turned, u)
    fresh = _whole(torch.where(fine[..., None], x, torch.zeros_like(x)).double(), s[..., None, None].expand_as(x)).clamp(-127, 127)
    new = is_new[..., None, :, None]
    u = torch.where(new, fresh, torch.where(is_old[..., None, :, None], u, torch.zeros_like(u)))
    marks = torch.where(is_new[..., None, :], ~fine, marks & is_old[..., None, :])
    return _blocks(u, s, marks, at)


def _values(blocks, at):
    """Stored values [..., 2, 16, D] in fp32."""
    s, marks = _params(blocks, at["k"].shape[-1])
    x = _codes(blocks, at).float() * s[..., None, None]
    return torch.where(marks[..., None], torch.full_like(x, math.nan), x)


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
        low = max(1, c["budget"] - c["budget"] // 8 if c["op"] == "evict" else length // 4)
        total[1:] = np.maximum(n[1:], r.randint(min(low, length), length + 1, b - 1))
    return total, n


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
    at = _places(dim, dev)
    pool = torch.zeros(count + spare, heads, page // 16, _block_bytes(c), dtype=torch.uint8, device=dev)
    # keys have channels of their own size and offset, values are plain; some tokens are larger than others
    size = torch.exp(0.5 * torch.randn(heads, dim, generator=gen, device=dev))
    mean = 0.5 * torch.randn(heads, dim, generator=gen, device=dev)

    def rows(n):
        k = torch.randn(n, heads, dim, generator=gen, device=dev) * size + mean
        v = torch.randn(n, heads, dim, generator=gen, device=dev)
        large = torch.exp(0.3 * torch.randn(n, heads, 1, generator=gen, device=dev))
        return (k * large).to(dtype), (v * large).to(dtype)

    held = lens - new if c["op"] == "write" else lens
    for i in range(b):  # the tokens that are in the cache before the call
        for first in range(0, int(held[i]), 16384):
            n = min(16384, int(held[i]) - first)
            blocks = torch.arange(first // 16, -(-(first + n) // 16), device=dev)
            x = torch.zeros(2, len(blocks) * 16, heads, dim, dtype=dtype, device=dev)
            x[0, :n], x[1, :n] = rows(n)
            x = x.unflatten(1, (-1, 16)).permute(1, 3, 0, 2, 4)                 # [blocks, H, 2, 16, D]
            is_new = (torch.arange(len(blocks) * 16, device=dev) < n).view(-1, 1, 16).expand(-1, heads, -1)
            where = table[i, blocks // (page // 16)].long(), slice(None), blocks % (page // 16)
            pool[where] = _write(pool[where], x, torch.zeros_like(is_new), is_new, at)
    starts = np.concatenate([[0], np.cumsum(new)])
    st = {"case": c, "pool": pool, "table": table, "at": at, "max_new": int(new.max()), "mass": None,
          "lens": torch.from_numpy(lens).int().to(dev), "starts": torch.from_numpy(starts).int().to(dev),
          "uniform": bool((new == new[0]).all()), "rows": int(starts[-1]), "scale": 1 / math.sqrt(dim)}
    if c["op"] in ("weigh", "evict"):  # the weight of earlier rows: a few tokens have most of it, the last have none yet
        mass = torch.exp(2 * torch.randn(pool.shape[0], heads, page, generator=gen, device=dev))
        st["mass"] = mass * (torch.rand(mass.shape, generator=gen, device=dev) > 0.05)
    if c["op"] == "write":
        st["k"], st["v"] = rows(st["rows"])
        # read back: the new rows and the up to 15 tokens before them whose block they joined
        st["back"] = torch.from_numpy(np.concatenate([[0], np.cumsum(new + 15)])).int().to(dev)
    elif c["op"] == "evict":
        st["kept"] = torch.empty(b, heads, c["budget"], dtype=torch.int32, device=dev)
        left = np.minimum(lens, c["budget"])
        st["left"] = torch.from_numpy(left).int().to(dev)
        st["back"] = torch.from_numpy(np.concatenate([[0], np.cumsum(left)])).int().to(dev)
    else:
        # queries lean on their key head's channels, so that scores are not all alike
        q = torch.randn(st["rows"], heads, c["q_heads"] // heads, dim, generator=gen, device=dev)
        q = q + 0.5 * torch.randn(st["rows"], heads, 1, dim, generator=gen, device=dev)
        st["q"] = q.flatten(1, 2).to(dtype)
    if "back" in st:
        counts = (new + 15) if c["op"] == "write" else np.minimum(lens, c["budget"])
        st["back_max"], st["back_rows"] = int(counts.max()), int(counts.sum())
    return st


# --------------------------------------------------------------------------- plain forms

def _positions(starts, lens, rows):
    """Sequence and position of every row, the last ones of each sequence."""
    starts, lens = starts.long(), lens.long()
    i = torch.arange(rows, device=starts.device)
    seq = torch.bucketize(i, starts[1:], right=True)
    return seq, lens[seq] - starts[seq + 1] + i


def _read(st, lens):
    """The stored rows `back`, in the cache's type; rows before a sequence's first token are zeros."""
    c, dtype = st["case"], _T[st["case"]["dtype"]]
    seq, pos = _positions(st["back"], lens, st["back_rows"])
    there, p = pos >= 0, pos.clamp_min(0)
    blocks = st["pool"][st["table"].long()[seq, p // c["page"]], :, p % c["page"] // 16]          # [N, H, bytes]
    s, marks = _params(blocks, c["dim"])
    t = p % 16
    pick = torch.stack((st["at"]["k"][t], st["at"]["v"][t]), 1)[:, None].expand(-1, c["kv_heads"], -1, -1)  # [N, H, 2, D]
    x = (blocks.gather(-1, pick.flatten(-2)).unflatten(-1, (2, -1)).float() - 128) * s[..., None]
    bad = marks.gather(-1, t[:, None, None, None].expand(-1, c["kv_heads"], 2, -1))
    x = torch.where(bad, torch.full_like(x, math.nan), x)
    x = torch.where(there[:, None, None, None], x, torch.zeros_like(x)).to(dtype)
    return {"k": x[:, :, 0].contiguous(), "v": x[:, :, 1].contiguous()}


def _plain_write(st):
    c = st["case"]
    dev, page, n = st["pool"].device, c["page"], st["max_new"]
    lens, starts = st["lens"].long(), st["starts"].long()
    first = lens - (starts[1:] - starts[:-1])                                    # the first new position
    most = (n + 14) // 16 + 1                                                    # blocks that a sequence's rows touch
    j = torch.minimum(first[:, None] // 16 + torch.arange(most, device=dev), (lens[:, None] - 1) // 16)  # the last again: the same twice
    pos = j[..., None] * 16 + torch.arange(16, device=dev)                       # [B, blocks, 16]
    is_old, is_new = pos < first[:, None, None], (pos >= first[:, None, None]) & (pos < lens[:, None, None])
    row = (starts[:-1, None, None] + pos - first[:, None, None]).clamp(0, st["rows"] - 1)
    x = torch.stack((st["k"][row], st["v"][row]), 2).permute(0, 1, 4, 2, 3, 5)   # [B, blocks, H, 2, 16, D]
    ids, sub = st["table"].long().gather(1, j // (page // 16)), j % (page // 16)
    every = (slice(None), slice(None), None)
    old = st["pool"][ids[..., None], torch.arange(c["kv_heads"], device=dev), sub[..., None]]
    st["pool"][ids[..., None], torch.arange(c["kv_heads"], device=dev), sub[..., None]] = _write(
        old, x, is_old[every].expand(-1, -1, c["kv_heads"], -1), is_new[every].expand(-1, -1, c["kv_heads"], -1), st["at"])
    return _read(st, st["lens"])


def _softmax_rows(s, seen):
    s = torch.where(seen, s, torch.full_like(s, -math.inf))
    top = s.amax(-1, keepdim=True)
    p = torch.exp(s - torch.where(torch.isfinite(top), top, torch.zeros_like(top)))
    total = p.sum(-1, keepdim=True)
    return p / torch.where(total > 0, total, torch.ones_like(total))


def _plain_attention(st):
    c, n = st["case"], st["max_new"]
    dev, heads = st["q"].device, c["kv_heads"]
    x = _values(st["pool"][st["table"].long().clamp_min(0)], st["at"])           # [B, pages, H, blocks, 2, 16, D]
    k, v = x.permute(4, 0, 2, 1, 3, 5, 6).flatten(3, 5)                          # [B, H, tokens, D]
    starts, lens = st["starts"].long(), st["lens"].long()
    j = torch.arange(n, device=dev)
    count = (starts[1:] - starts[:-1])[:, None]
    i = (starts[:-1, None] + j).clamp_max(st["rows"] - 1)                        # [B, n]: every sequence padded to n rows
    last = lens[:, None] - count + j                                             # position of each row
    q = st["q"].float()[i].unflatten(2, (heads, -1)).permute(0, 2, 1, 3, 4)      # [B, H, n, g, D]
    shape = q.shape
    s = q.flatten(2, 3) @ k.transpose(-1, -2) * st["scale"]
    seen = (torch.arange(k.shape[2], device=dev) <= last[:, :, None]) & (j < count)[:, :, None]
    seen = seen[:, None, :, None, :].expand(-1, 1, -1, shape[3], -1).flatten(2, 3)
    p = _softmax_rows(s, seen)
    o = (p @ v).view(shape).permute(0, 2, 1, 3, 4).flatten(2, 3)
    seq, _ = _positions(st["starts"], st["lens"], st["rows"])
    out = {"out": o[seq, torch.arange(st["rows"], device=dev) - starts[seq]].to(st["q"].dtype)}
    if c["op"] == "weigh":
        got = p.sum(2).unflatten(2, (-1, c["page"])).transpose(1, 2)             # [B, pages, H, page]; nothing beyond a sequence
        pages = st["table"].long()
        got = torch.where((pages >= 0)[..., None, None], got, torch.zeros_like(got))
        st["mass"].index_add_(0, pages.clamp_min(0).flatten(), got.flatten(0, 1))
        out["mass"] = st["mass"]
    return out


def _plain_kept(st):
    """[B, H, budget]: the positions that stay, ascending, -1 after them."""
    c = st["case"]
    pages, lens = st["table"].long().clamp_min(0), st["lens"].long()[:, None, None]
    mass = st["mass"][pages].transpose(1, 2).flatten(2, 3)                       # [B, H, tokens]
    mass = torch.where(torch.isnan(mass), torch.full_like(mass, -math.inf), mass)
    j = torch.arange(mass.shape[2], device=mass.device)
    rank = torch.where((j < c["first"]) | (j >= lens - c["last"]), 2, 1).expand_as(mass)  # always, by mass, never
    rank = torch.where(j < lens, rank, torch.zeros_like(rank))
    by_mass = torch.sort(mass, dim=-1, descending=True, stable=True).indices
    order = torch.sort(rank.gather(-1, by_mass), dim=-1, descending=True, stable=True).indices
    pick = by_mass.gather(-1, order)[..., :c["budget"]]
    none = torch.full_like(pick, 1 << 40)
    pick = torch.sort(torch.where(pick < lens, pick, none), -1).values
    short = torch.full(pick.shape[:2] + (c["budget"] - pick.shape[2],), 1 << 40, device=pick.device)
    pick = torch.cat((pick, short), -1)
    return torch.where(pick < (1 << 40), pick, torch.full_like(pick, -1))


def _plain_evict(st):
    c = st["case"]
    dev, page, heads = st["pool"].device, c["page"], c["kv_heads"]
    kept = _plain_kept(st)
    many = -(-c["budget"] // 16) * 16
    src = torch.cat((kept, torch.full(kept.shape[:2] + (many - c["budget"],), -1, device=dev)), -1)  # [B, H, whole blocks]
    there, p = src >= 0, src.clamp_min(0)
    h = torch.arange(heads, device=dev)[None, :, None]
    ids = st["table"].long().clamp_min(0)[torch.arange(c["batch"], device=dev)[:, None, None], p // page]
    blocks = st["pool"][ids, h, p % page // 16]                                  # [B, H, tokens, bytes]
    s, marks = _params(blocks, c["dim"])
    t = p % 16
    pick = torch.stack((st["at"]["k"][t], st["at"]["v"][t]), 3)                  # [B, H, tokens, 2, D]
    u = blocks.gather(-1, pick.flatten(-2)).unflatten(-1, (2, -1)).int() - 128
    bad = marks.gather(-1, t[..., None, None].expand(-1, -1, -1, 2, -1))[..., 0]  # [B, H, tokens, 2]
    s = torch.where(there[..., None], s, torch.zeros_like(s))
    by16 = lambda x: x.unflatten(2, (-1, 16)).transpose(3, 4)                    # noqa: E731  [B, H, blocks, 2, 16, ..]
    u, s, bad = by16(u), by16(s), by16(bad & there[..., None])
    to = s.amax(-1)
    u = torch.where((s == to[..., None])[..., None], u, _whole(u.double() * s.double()[..., None], to[..., None, None].expand_as(u)))
    # what stays of blocks: those of no kept token, and of a last block the bytes of tokens beyond the budget
    j = torch.arange(many // 16, device=dev).clamp_max(st["table"].shape[1] * (page // 16) - 1)
    into = st["table"].long()[:, None, j // (page // 16)]
    live = there.unflatten(2, (-1, 16)).any(-1) & (into >= 0)
    spare = st["pool"].shape[0]
    pool = torch.cat((st["pool"], torch.empty_like(st["pool"][:1])))             # a page that takes what is written nowhere
    pool[torch.where(live, into, torch.full_like(into, spare)), h, j % (page // 16)] = _blocks(u, to, bad, st["at"])
    st["pool"].copy_(pool[:spare])
    j = torch.arange(c["budget"], device=dev).clamp_max(st["table"].shape[1] * page - 1)
    into = st["table"].long()[:, None, j // page].expand(-1, heads, -1)
    mass = torch.cat((st["mass"], torch.empty_like(st["mass"][:1])))
    mass[torch.where(kept >= 0, into, torch.full_like(into, spare)), h, j % page] = st["mass"][ids, h, p % page][..., :c["budget"]]
    st["mass"].copy_(mass[:spare])
    return {"kept": kept.int(), "mass": st["mass"], **_read(st, st["left"])}


_PLAIN = {"write": _plain_write, "attention": _plain_attention, "weigh": _plain_attention, "evict": _plain_evict}


def run(state):
    c = state["case"]
    if not own:
        return _PLAIN[c["op"]](state)
    cache = state.get("cache")
    if cache is None:  # the handle that a program makes once
        from moe_expert_layer_sorted_gb300 import KVCache8
        cache = state["cache"] = KVCache8(state["pool"], page_size=c["page"], head_dim=c["dim"], dtype=_T[c["dtype"]],
                                          mass=state["mass"])
    batch = dict(table=state["table"], lens=state["lens"])
    ragged = dict(starts=state["starts"], max_new=state["max_new"])
    shape = (state["rows"],)
    if state["uniform"]:
        shape, ragged = (c["batch"], state["max_new"]), {}
    if c["op"] in ("write", "evict"):
        out = {}
        if c["op"] == "write":
            cache.append(state["k"].view(*shape, *state["k"].shape[1:]), state["v"].view(*shape, *state["v"].shape[1:]),
                         **batch, **ragged)
        else:
            cache.evict(state["kept"], keep_first=c["first"], keep_last=c["last"], **batch)
            out = {"kept": state["kept"], "mass": state["mass"]}
            batch["lens"] = state["left"]
        k, v = (torch.empty(state["back_rows"], c["kv_heads"], c["dim"], dtype=_T[c["dtype"]], device=state["pool"].device)
                for _ in range(2))
        cache.read(k, v, starts=state["back"], max_new=state["back_max"], **batch)
        return {**out, "k": k, "v": v}
    q = state["q"].view(*shape, *state["q"].shape[1:])
    out = torch.empty_like(state["q"])
    if c["op"] == "attention":
        cache.attention(q, out.view(q.shape), scale=state["scale"], **batch, **ragged)
        return {"out": out}
    lse = torch.empty(state["rows"], c["q_heads"], device=out.device)
    cache.attention(q, out.view(q.shape), scale=state["scale"], lse=lse, weigh=True, **batch, **ragged)
    return {"out": out, "mass": state["mass"]}


def work(case):
    """Every input once, every output once; a stored row and head takes 2 D + 1 bytes."""
    c = case
    lens, new = (x.astype(np.float64) for x in _lengths(c))
    row = c["kv_heads"] * (2.0 * c["dim"] + 1)
    wide = 4.0 * c["kv_heads"] * c["dim"]                # a row's keys and values in 16 bits
    qo = 4.0 * c["q_heads"] * c["dim"]                   # a row's queries and outputs
    n = float(new.sum())
    if c["op"] == "write":                               # written, and read back with the tokens before
        m = n + 15 * c["batch"]
        return {"bytes": n * (wide + row) + m * (row + wide), "flops": 2.0 * (n + m) * wide}
    if c["op"] == "evict":                               # masses read, kept rows read and written, and read back
        left = np.minimum(lens, c["budget"])
        moved = float(left[lens > c["budget"]].sum())
        return {"bytes": 4.0 * c["kv_heads"] * float(lens.sum()) + moved * (2 * row + 8.0 * c["kv_heads"])
                + 4.0 * c["kv_heads"] * c["budget"] * c["batch"] + float(left.sum()) * (row + wide),
                "flops": 2.0 * float(lens.sum()) * c["kv_heads"] + (moved + float(left.sum())) * wide}
    seen = float((new * lens - new * (new - 1) / 2).sum())  # visible (row, token) pairs
    tokens = float(lens.sum())
    return {"bytes": tokens * row + n * qo + (8.0 * tokens * c["kv_heads"] if c["op"] == "weigh" else 0.0),
            "flops": 4.0 * c["q_heads"] * c["dim"] * seen + (c["q_heads"] * seen if c["op"] == "weigh" else 0.0)}


# ------------------------------------------------------------- the definition in 64 bits

def exact(case, seed):
    """Block by block and row by row from the definition, in 64 bits; which tokens stay is a
    whole-number output and has none."""
    st = prepare(case, seed)
    c, dtype = st["case"], _T[case["dtype"]]
    dev, heads, dim, page = st["pool"].device, c["kv_heads"], c["dim"], c["page"]
    lens, starts = st["lens"].tolist(), st["starts"].tolist()
    d, tok = np.arange(dim)[None], np.arange(16)[:, None]
    pair = tok // 2 % 4
    kbyte = tok * dim + (d // 16 * 16 ^ (64 * (tok % 2) if dim == 128 else 0 * tok)) + d % 16
    vbyte = tok // 2 * 2 * dim + (d // 8 * 16 ^ (16 * (pair % 2) + 64 * (pair // 2) if dim == 128 else 32 * pair)) + d % 8 * 2 + tok % 2
    kbyte, vbyte = torch.from_numpy(kbyte).to(dev), torch.from_numpy(16 * dim + vbyte).to(dev)

    def held(b, h, pos):
        """Codes and steps of the keys and values of positions pos of sequence b's head h."""
        block = st["pool"][st["table"][b].long()[pos // page], h, pos % page // 16]
        step = block[:, 32 * dim:32 * dim + 8].contiguous().view(torch.float32).double()
        return [(block.gather(1, byte[pos % 16]).double() - 128, step[:, side]) for side, byte in ((0, kbyte), (1, vbyte))]

    def settle(u, s, to):
        """Codes u of steps s, turned to step `to` and read."""
        safe = torch.where(to > 0, to, torch.ones_like(to))
        return torch.where((s == to)[:, None], u, (u * s[:, None] / safe[:, None]).round()) * to[:, None]

    if c["op"] in ("write", "evict"):
        kv = torch.zeros(2, st["back_rows"], heads, dim, dtype=torch.float64, device=dev)
        back, kept = st["back"].tolist(), _plain_kept(st) if c["op"] == "evict" else None
        for b in range(c["batch"]):
            for h in range(heads):
                if c["op"] == "evict":
                    pos = kept[b, h][kept[b, h] >= 0]
                    for side, (u, s) in enumerate(held(b, h, pos)):
                        pad = torch.zeros(-(-len(pos) // 16) * 16, dtype=torch.float64, device=dev)
                        pad[:len(pos)] = s
                        to = pad.view(-1, 16).max(1).values.repeat_interleave(16)[:len(pos)]
                        kv[side, back[b]:back[b + 1], h] = settle(u, s, to)
                    continue
                n = starts[b + 1] - starts[b]
                first = lens[b] - n
                lo = first // 16 * 16
                have = max(0, first - 15)
                older = torch.arange(lo, first, device=dev)
                pos = torch.arange(have, first, device=dev)
                was = held(b, h, older) if first > lo else None
                for side, (src, (u, s)) in enumerate(zip((st["k"], st["v"]), held(b, h, pos) if first else [(None, None)] * 2)):
                    x = torch.zeros(-(-lens[b] // 16) * 16 - lo, dim, dtype=torch.float64, device=dev)
                    x[first - lo:lens[b] - lo] = src[starts[b]:starts[b + 1], h].double()
                    step = (x.abs().view(-1, 16 * dim).max(1).values / 127).float().double()
                    if was is not None:
                        step[0] = torch.maximum(step[0], was[side][1][0])
                    to = step.repeat_interleave(16)
                    safe = torch.where(to > 0, to, torch.ones_like(to))
                    fresh = (x / safe[:, None]).round().clamp(-127, 127) * to[:, None]
                    end = back[b + 1]
                    kv[side, end - n:end, h] = fresh[first - lo:lens[b] - lo]
                    if first:
                        now = torch.where(pos >= lo, step[0], s)
                        kv[side, end - n - len(pos):end - n, h] = settle(u, s, now)
        out = {"k": kv[0], "v": kv[1]}
        if c["op"] == "evict":
            mass = st["mass"].double()
            for b in range(c["batch"]):
                for h in range(heads):
                    pos = kept[b, h][kept[b, h] >= 0]
                    j = torch.arange(len(pos), device=dev)
                    ids = st["table"][b].long()
                    mass[ids[j // page], h, j % page] = st["mass"][ids[pos // page], h, pos % page].double()
            out.update(kept=None, mass=mass)
        return out
    per = c["q_heads"] // heads
    out = torch.zeros(st["rows"], c["q_heads"], dim, dtype=torch.float64, device=dev)
    mass = st["mass"].double() if c["op"] == "weigh" else None
    for b in range(c["batch"]):
        n = starts[b + 1] - starts[b]
        pos = torch.arange(lens[b], device=dev)
        for h in range(heads):
            k, v = (u * s[:, None] for u, s in held(b, h, pos))
            total = torch.zeros(lens[b], dtype=torch.float64, device=dev)
            for a in range(0, n, 1024):
                z = min(n, a + 1024)
                q = st["q"][starts[b] + a:starts[b] + z, h * per:(h + 1) * per].double()
                s = torch.einsum("ngd,ld->ngl", q, k) / math.sqrt(dim)
                hidden = pos[None, :] > lens[b] - n + torch.arange(a, z, device=dev)[:, None]
                w = torch.softmax(s.masked_fill(hidden[:, None], -math.inf), -1)
                out[starts[b] + a:starts[b] + z, h * per:(h + 1) * per] = torch.einsum("ngl,ld->ngd", w, v)
                total += w.sum((0, 1))
            if mass is not None:
                mass[st["table"][b].long()[pos // page], h, pos % page] += total
    return {"out": out} if mass is None else {"out": out, "mass": mass}
