"""The 4-bit key/value cache (see moe_kv_* in include/moe.h): argument checks and
marshalling; the work is done in the CUDA library."""
from __future__ import annotations

import ctypes
import math
import struct

_P = ctypes.c_void_p
_I64 = ctypes.c_int64
KV_BF16, KV_F16 = 0, 1


class KVDesc(ctypes.Structure):
    _fields_ = [("struct_size", ctypes.c_uint32), ("device", ctypes.c_int32), ("dtype", ctypes.c_int32),
                ("num_layers", ctypes.c_int32), ("kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32),
                ("group_size", ctypes.c_int32), ("page_size", ctypes.c_int32), ("num_pages", _I64),
                ("pages", _P), ("bounds", _P), ("reserved", _I64 * 2)]


# moe_kv_batch and moe_kv_tensor, packed
_BATCH = struct.Struct("=I3i2q3Q")
_BATCH_SIZE = _BATCH.size
_TENSOR = struct.Struct("=Q3q")


def declare(L):
    """Argument types of the library's moe_kv_* functions."""
    i32, B, X = ctypes.c_int, ctypes.c_char_p, ctypes.c_char_p  # packed structures
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
        self._lib = _lib()
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
        rc = self._lib.moe_kv_create(ctypes.byref(d), ctypes.byref(h))
        if rc:
            raise MoeError(rc, self._lib.moe_kv_last_error(None).decode())
        self._h, self.pages, self.bounds, self.desc = h, pages, bounds, d
        self.dtype, self.device = dtype, pages.device
        self.layers, self.kv_heads, self.head_dim = layers, kv_heads, head_dim
        self.page_size, self.group_size = page_size, group_size
        self._scale = 1.0 / math.sqrt(head_dim)
        self._index, self._i32 = pages.device.index, torch.int32
        self._current_stream = torch._C._cuda_getCurrentRawStream

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
            self._lib.moe_kv_destroy(self._h)
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    # ------------------------------------------------------------------ marshalling
    # A decode step's calls are a few microseconds of GPU work each, so the host's share
    # counts: the C structures are packed in one step each, and tensors are asked for
    # nothing twice.

    def _int(self, t, name, dim):
        if not (t.dtype is self._i32 and t.is_cuda and t.get_device() == self._index and t.dim() == dim):
            _bad(f"{name}: int32 tensor of {dim} axes on {self.device}")
        return t.data_ptr()

    def _batch(self, shape, table, lens, starts, max_new):
        tp, lp, sp = self._int(table, "table", 2), self._int(lens, "lens", 1), 0
        n, (sequences, cols) = len(shape), table.shape
        batch = lens.shape[0]
        if sequences != batch:
            _bad("table and lens name different numbers of sequences")
        stride, step = table.stride()
        if (step != 1 and cols > 1) or (batch > 1 and lens.stride(0) != 1):
            _bad("table's rows and lens must be contiguous")
        if batch <= 1:
            stride = cols
        if starts is None:
            if n != 4 or shape[0] != batch:
                _bad("row tensors without starts: [sequences, rows, heads, head_dim]")
            if max_new is not None and max_new != shape[1]:
                _bad("max_new belongs to starts")
            max_new = shape[1]
            rows = batch * max_new
        else:
            if n != 3:
                _bad("row tensors with starts: [rows, heads, head_dim]")
            sp = self._int(starts, "starts", 1)
            if starts.shape[0] != batch + 1 or starts.stride(0) != 1:
                _bad("starts: contiguous, one entry more than sequences")
            rows = shape[0]
            if max_new is None:
                max_new = rows
        if not (0 <= max_new < 1 << 31 and rows < 1 << 62 and batch < 1 << 31 and cols < 1 << 31):
            _bad("max_new, the sequences or the table's pages are out of range")
        return rows, _BATCH.pack(_BATCH_SIZE, batch, max_new, cols, stride, rows, tp, lp, sp)

    def _rows(self, t, name, shape, written=False):
        if not (t.dtype is self.dtype and t.is_cuda and t.get_device() == self._index and t.shape == shape):
            _bad(f"{name}: {self.dtype} on {self.device}, expected shape {tuple(shape)}")
        st = t.stride()
        if written and 0 in st and any(n > 1 and d == 0 for n, d in zip(shape, st)):
            _bad(f"{name}: an expanded tensor cannot be written to")
        if st[-1] != 1:
            _bad(f"{name}: the channels must be contiguous")
        if len(shape) == 4:
            b, r, h, _ = st
            nb, nr, nh, _ = shape
            # axes of length 1 have no stride that matters
            return _TENSOR.pack(t.data_ptr(), b if nb > 1 else 0, r if nr > 1 else 0, h if nh > 1 else 0)
        r, h, _ = st
        return _TENSOR.pack(t.data_ptr(), 0, r if shape[0] > 1 else 0, h if shape[1] > 1 else 0)

    def _heads(self, shape, name, kv):
        if not (3 <= len(shape) <= 4 and shape[-1] == self.head_dim and (not kv or shape[-2] == self.kv_heads)):
            _bad(f"{name}: [..., {self.kv_heads if kv else 'heads'}, {self.head_dim}] with 3 or 4 axes, got {tuple(shape)}")
        return shape[-2]

    def _failed(self, rc):
        from . import MoeError
        # a busy handle's text is the running call's
        raise MoeError(rc, "the cache is in use by another thread" if rc == 5 else
                       self._lib.moe_kv_last_error(self._h).decode())

    def _stream(self, stream):
        if stream is None:
            return self._current_stream(self._index)
        return stream if isinstance(stream, int) else stream.cuda_stream

    # ------------------------------------------------------------------------- calls

    def append(self, k, v, *, table, lens, starts=None, max_new=None, layer=0, stream=None):
        """Quantise the rows k, v into the sequences' pages and update the pages' bounds."""
        shape = k.shape
        self._heads(shape, "k", True)
        _, b = self._batch(shape, table, lens, starts, max_new)
        rc = self._lib.moe_kv_append(self._h, layer, b, self._rows(k, "k", shape), self._rows(v, "v", shape),
                                     self._stream(stream))
        if rc:
            self._failed(rc)

    def read(self, k, v, *, table, lens, starts=None, max_new=None, layer=0, stream=None):
        """The stored keys and values of the rows, into k and v."""
        shape = k.shape
        self._heads(shape, "k", True)
        _, b = self._batch(shape, table, lens, starts, max_new)
        rc = self._lib.moe_kv_read(self._h, layer, b, self._rows(k, "k", shape, True), self._rows(v, "v", shape, True),
                                   self._stream(stream))
        if rc:
            self._failed(rc)

    def attention(self, q, out, *, table, lens, starts=None, max_new=None, scale=None, causal=True, lse=None,
                  pages=None, layer=0, stream=None):
        """out = softmax(scale q k^T) v of the rows q (scale None: 1 / sqrt(head_dim)).
        pages: None, or `select`'s choice, the only pages then attended to.  lse: None, or
        float32 [rows, heads] for the logarithm of each row's sum of exponentials."""
        shape = q.shape
        heads = self._heads(shape, "q", False)
        rows, b = self._batch(shape, table, lens, starts, max_new)
        lp = pp = None
        budget = 0
        if lse is not None:
            import torch
            if not (lse.device == self.device and lse.dtype == torch.float32 and lse.is_contiguous()
                    and lse.numel() == rows * heads):
                _bad("lse: contiguous float32, one value per row and query head")
            lp = lse.data_ptr()
        if pages is not None:
            budget = self._choice(pages, rows)
            pp = pages.data_ptr()
        rc = self._lib.moe_kv_attention(self._h, layer, b, self._rows(q, "q", shape), heads,
                                        self._scale if scale is None else scale, 1 if causal else 0,
                                        self._rows(out, "out", shape, True), lp, pp, budget, self._stream(stream))
        if rc:
            self._failed(rc)

    def _choice(self, pages, rows):
        if not (pages.dtype is self._i32 and pages.is_cuda and pages.get_device() == self._index and pages.is_contiguous()
                and pages.dim() >= 3 and pages.shape[-2] == self.kv_heads
                and pages.numel() == rows * self.kv_heads * pages.shape[-1]):
            _bad("pages: contiguous int32 [rows, kv_heads, budget]")
        return pages.shape[-1]

    def select(self, q, pages, *, table, lens, starts=None, max_new=None, keep_first=1, keep_last=1, layer=0,
               stream=None):
        """Choose pages.shape[-1] pages for each row and kv head into pages (int32 [rows,
        kv_heads, budget], ascending, -1 where a row sees fewer): the first keep_first, the
        last keep_last, then those whose bounds promise the largest q . k."""
        shape = q.shape
        heads = self._heads(shape, "q", False)
        rows, b = self._batch(shape, table, lens, starts, max_new)
        rc = self._lib.moe_kv_select(self._h, layer, b, self._rows(q, "q", shape), heads, self._choice(pages, rows),
                                     keep_first, keep_last, pages.data_ptr(), self._stream(stream))
        if rc:
            self._failed(rc)
