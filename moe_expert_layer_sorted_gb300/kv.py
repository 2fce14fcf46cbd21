"""The 4-bit key/value cache (see moe_kv_* in include/moe.h): argument checks and
marshalling; the work is done in the CUDA library."""
from __future__ import annotations

import ctypes
import math

_P = ctypes.c_void_p
_I64 = ctypes.c_int64
KV_BF16, KV_F16 = 0, 1


class KVDesc(ctypes.Structure):
    _fields_ = [("struct_size", ctypes.c_uint32), ("device", ctypes.c_int32), ("dtype", ctypes.c_int32),
                ("num_layers", ctypes.c_int32), ("kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32),
                ("group_size", ctypes.c_int32), ("page_size", ctypes.c_int32), ("num_pages", _I64),
                ("pages", _P), ("bounds", _P), ("reserved", _I64 * 2)]


class KVBatch(ctypes.Structure):
    _fields_ = [("struct_size", ctypes.c_uint32), ("batch", ctypes.c_int32), ("max_new", ctypes.c_int32),
                ("table_pages", ctypes.c_int32), ("table_stride", _I64), ("rows", _I64),
                ("table", _P), ("lens", _P), ("starts", _P)]


class KVTensor(ctypes.Structure):
    _fields_ = [("data", _P), ("batch_stride", _I64), ("row_stride", _I64), ("head_stride", _I64)]


def declare(L):
    """Argument types of the library's moe_kv_* functions."""
    i32, B, X = ctypes.c_int, ctypes.POINTER(KVBatch), ctypes.POINTER(KVTensor)
    L.moe_kv_sizes.argtypes = [ctypes.POINTER(KVDesc), ctypes.POINTER(_I64), ctypes.POINTER(_I64)]
    L.moe_kv_create.argtypes = [ctypes.POINTER(KVDesc), ctypes.POINTER(_P)]
    L.moe_kv_destroy.argtypes = [_P]
    L.moe_kv_append.argtypes = [_P, i32, B, X, X, _P]
    L.moe_kv_read.argtypes = [_P, i32, B, X, X, _P]
    L.moe_kv_attention.argtypes = [_P, i32, B, X, i32, ctypes.c_float, i32, X, _P, _P, i32, _P]
    L.moe_kv_select.argtypes = [_P, i32, B, X, i32, i32, i32, i32, _P, _P]
    L.moe_kv_last_error.argtypes = [_P]
    L.moe_kv_last_error.restype = ctypes.c_char_p


def _lib():
    from . import lib
    return lib()


def _bad(msg):
    from . import MoeError
    raise MoeError(1, msg)


def _desc(dtype, num_layers, kv_heads, head_dim, group_size, page_size, num_pages):
    import torch
    if dtype not in (torch.bfloat16, torch.float16):
        _bad("dtype must be torch.bfloat16 or torch.float16")
    d = KVDesc()
    d.struct_size = ctypes.sizeof(KVDesc)
    d.dtype = KV_BF16 if dtype == torch.bfloat16 else KV_F16
    d.num_layers, d.kv_heads, d.head_dim, d.group_size = num_layers, kv_heads, head_dim, group_size
    d.page_size, d.num_pages = page_size, num_pages
    return d


class KVCache:
    """A paged key/value cache in 4 bits for `num_layers` layers, with what writes it,
    reads it, attends over it and chooses its pages.

    pages: uint8 CUDA tensor [num_pages, kv_heads, page_size / 16, block bytes], or with a
    leading layer axis; contiguous.  bounds: None, or a tensor of the cache's dtype
    [num_pages, kv_heads, 2, head_dim] with the same leading axis, which `append` keeps and
    `select` needs.  `KVCache.allocate` makes both.

    A batch of sequences is given to each call by
      table   int32 [sequences, pages]: the pages of each sequence in order (rows may be strided);
      lens    int32 [sequences]: tokens in the cache, the call's own rows included;
      starts  None: tensors are [sequences, rows, heads, head_dim], the rows being the last
              tokens of each sequence.  int32 [sequences + 1]: tensors are [rows, heads,
              head_dim], rows starts[s] .. starts[s + 1] being sequence s's; max_new is then
              the most rows of any sequence (None: all rows).
    These are CUDA tensors and are read on the device only.  Row tensors may be strided
    (16-byte aligned rows and heads, contiguous channels).  Work goes to `stream` (None:
    torch's current stream)."""

    def __init__(self, pages, *, page_size, head_dim, group_size=64, dtype=None, bounds=None):
        import torch
        from . import MoeError
        self._h = None
        dtype = torch.bfloat16 if dtype is None else dtype
        if not (pages.is_cuda and pages.dtype == torch.uint8 and pages.dim() in (4, 5) and pages.is_contiguous()):
            _bad("pages: contiguous uint8 CUDA tensor [layers,] num_pages, kv_heads, blocks, block bytes")
        shape = tuple(pages.shape)
        layers = shape[0] if len(shape) == 5 else 1
        num_pages, kv_heads = shape[-4], shape[-3]
        d = _desc(dtype, layers, kv_heads, head_dim, group_size, page_size, num_pages)
        want = (num_pages, kv_heads) + self._block_shape(head_dim, group_size, page_size)
        if shape[-4:] != want:
            _bad(f"pages: trailing shape {shape[-4:]}, expected {want}")
        if bounds is not None:
            if not (bounds.device == pages.device and bounds.dtype == dtype and bounds.is_contiguous()
                    and tuple(bounds.shape) == shape[:-4] + (num_pages, kv_heads, 2, head_dim)):
                _bad("bounds: contiguous [layers,] num_pages, kv_heads, 2, head_dim of the cache's dtype")
        d.device = pages.device.index
        d.pages = pages.data_ptr()
        d.bounds = None if bounds is None else bounds.data_ptr()
        h = _P()
        rc = _lib().moe_kv_create(ctypes.byref(d), ctypes.byref(h))
        if rc:
            raise MoeError(rc, _lib().moe_kv_last_error(None).decode())
        self._h, self.pages, self.bounds, self.desc = h, pages, bounds, d
        self.dtype, self.device = dtype, pages.device
        self.layers, self.kv_heads, self.head_dim = layers, kv_heads, head_dim
        self.page_size, self.group_size = page_size, group_size
        self._scale = 1.0 / math.sqrt(head_dim)

    @staticmethod
    def _block_shape(head_dim, group_size, page_size):
        if group_size < 1 or page_size < 16:
            _bad("group_size and page_size must be positive multiples of 32 and 16")
        return page_size // 16, 16 * (head_dim + 8 * (head_dim // group_size))

    @classmethod
    def allocate(cls, num_pages, *, kv_heads, head_dim, page_size=64, group_size=64, dtype=None, layers=1,
                 bounds=True, device="cuda"):
        """A cache with pages (and bounds) of its own."""
        import torch
        dtype = torch.bfloat16 if dtype is None else dtype
        shape = (layers, num_pages, kv_heads)
        pages = torch.empty(shape + cls._block_shape(head_dim, group_size, page_size), dtype=torch.uint8, device=device)
        ends = torch.zeros(shape + (2, head_dim), dtype=dtype, device=device) if bounds else None
        return cls(pages, page_size=page_size, head_dim=head_dim, group_size=group_size, dtype=dtype, bounds=ends)

    def close(self):
        if getattr(self, "_h", None):
            _lib().moe_kv_destroy(self._h)
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    # ------------------------------------------------------------------ marshalling

    def _int(self, t, name, dim):
        import torch
        if not (t.device == self.device and t.dtype == torch.int32 and t.dim() == dim and (t.shape[-1] < 2 or t.stride(-1) == 1)):
            _bad(f"{name}: int32 tensor of {dim} axes on {self.device}, its last axis contiguous")
        return t.data_ptr()

    def _batch(self, shape, table, lens, starts, max_new):
        b = KVBatch()
        b.struct_size = ctypes.sizeof(KVBatch)
        b.table, b.lens = self._int(table, "table", 2), self._int(lens, "lens", 1)
        b.batch = lens.shape[0]
        if table.shape[0] != b.batch:
            _bad("table and lens name different numbers of sequences")
        b.table_pages = table.shape[1]
        b.table_stride = table.stride(0) if b.batch > 1 else table.shape[1]
        if starts is None:
            if len(shape) != 4 or shape[0] != b.batch:
                _bad("row tensors without starts: [sequences, rows, heads, head_dim]")
            if max_new is not None and max_new != shape[1]:
                _bad("max_new belongs to starts")
            b.max_new, b.rows = shape[1], shape[0] * shape[1]
        else:
            if len(shape) != 3:
                _bad("row tensors with starts: [rows, heads, head_dim]")
            b.starts = self._int(starts, "starts", 1)
            if starts.shape[0] != b.batch + 1:
                _bad("starts: one entry more than sequences")
            b.rows = shape[0]
            b.max_new = shape[0] if max_new is None else max_new
        return b

    def _rows(self, t, name, shape=None, written=False):
        if not (t.device == self.device and t.dtype == self.dtype and t.dim() in (3, 4) and t.shape[-1] == self.head_dim
                and t.stride(-1) == 1):
            _bad(f"{name}: {self.dtype} on {self.device}, [..., heads, {self.head_dim}] with contiguous channels")
        if shape is not None and t.shape != shape:
            _bad(f"{name}: shape {tuple(t.shape)}, expected {tuple(shape)}")
        st = t.stride()
        if written and any(n > 1 and d == 0 for n, d in zip(t.shape, st)):
            _bad(f"{name}: an expanded tensor cannot be written to")
        x = KVTensor()
        # axes of length 1 have no stride that matters
        x.data, x.head_stride = t.data_ptr(), st[-2] if t.shape[-2] > 1 else 0
        x.row_stride = st[-3] if t.shape[-3] > 1 else 0
        x.batch_stride = st[0] if t.dim() == 4 and t.shape[0] > 1 else 0
        return x

    def _call(self, rc):
        if rc:
            from . import MoeError
            # a busy handle's text is the running call's
            raise MoeError(rc, "the cache is in use by another thread" if rc == 5 else
                           _lib().moe_kv_last_error(self._h).decode())

    def _stream(self, stream):
        if stream is None:
            import torch
            return torch.cuda.current_stream(self.device).cuda_stream
        return stream if isinstance(stream, int) else stream.cuda_stream

    # ------------------------------------------------------------------------- calls

    def append(self, k, v, *, table, lens, starts=None, max_new=None, layer=0, stream=None):
        """Quantise the rows k, v into the sequences' pages and update the pages' bounds."""
        if k.shape[-2] != self.kv_heads:
            _bad(f"k: {k.shape[-2]} heads, the cache has {self.kv_heads}")
        b = self._batch(k.shape, table, lens, starts, max_new)
        kt, vt = self._rows(k, "k"), self._rows(v, "v", k.shape)
        self._call(_lib().moe_kv_append(self._h, layer, ctypes.byref(b), ctypes.byref(kt), ctypes.byref(vt),
                                        self._stream(stream)))

    def read(self, k, v, *, table, lens, starts=None, max_new=None, layer=0, stream=None):
        """The stored keys and values of the rows, into k and v."""
        if k.shape[-2] != self.kv_heads:
            _bad(f"k: {k.shape[-2]} heads, the cache has {self.kv_heads}")
        b = self._batch(k.shape, table, lens, starts, max_new)
        kt, vt = self._rows(k, "k", written=True), self._rows(v, "v", k.shape, written=True)
        self._call(_lib().moe_kv_read(self._h, layer, ctypes.byref(b), ctypes.byref(kt), ctypes.byref(vt),
                                      self._stream(stream)))

    def attention(self, q, out, *, table, lens, starts=None, max_new=None, scale=None, causal=True, lse=None,
                  pages=None, layer=0, stream=None):
        """out = softmax(scale q k^T) v of the rows q (scale None: 1 / sqrt(head_dim)).
        pages: None, or `select`'s choice, the only pages then attended to.  lse: None, or
        float32 [rows, heads] for the logarithm of each row's sum of exponentials."""
        import torch
        b = self._batch(q.shape, table, lens, starts, max_new)
        qt, ot = self._rows(q, "q"), self._rows(out, "out", q.shape, written=True)
        lp = pp = None
        budget = 0
        if lse is not None:
            if not (lse.device == self.device and lse.dtype == torch.float32 and lse.is_contiguous()
                    and lse.numel() == b.rows * q.shape[-2]):
                _bad("lse: contiguous float32, one value per row and query head")
            lp = lse.data_ptr()
        if pages is not None:
            budget = self._choice(pages, b)
            pp = pages.data_ptr()
        self._call(_lib().moe_kv_attention(self._h, layer, ctypes.byref(b), ctypes.byref(qt), q.shape[-2],
                                           self._scale if scale is None else scale, int(causal), ctypes.byref(ot), lp,
                                           pp, budget, self._stream(stream)))

    def _choice(self, pages, b):
        import torch
        if not (pages.device == self.device and pages.dtype == torch.int32 and pages.is_contiguous() and pages.dim() >= 3
                and pages.shape[-2] == self.kv_heads and pages.numel() == b.rows * self.kv_heads * pages.shape[-1]):
            _bad("pages: contiguous int32 [rows, kv_heads, budget]")
        return pages.shape[-1]

    def select(self, q, pages, *, table, lens, starts=None, max_new=None, keep_first=1, keep_last=1, layer=0,
               stream=None):
        """Choose pages.shape[-1] pages for each row and kv head into pages (int32 [rows,
        kv_heads, budget], ascending, -1 where a row sees fewer): the first keep_first, the
        last keep_last, then those whose bounds promise the largest q . k."""
        b = self._batch(q.shape, table, lens, starts, max_new)
        qt = self._rows(q, "q")
        budget = self._choice(pages, b)
        self._call(_lib().moe_kv_select(self._h, layer, ctypes.byref(b), ctypes.byref(qt), q.shape[-2], budget,
                                        keep_first, keep_last, pages.data_ptr(), self._stream(stream)))
