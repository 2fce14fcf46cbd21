"""The 4-bit key/value cache (see moe_kv_* in include/moe.h): the handle and its
tensors; the work is done in the CUDA library."""
from __future__ import annotations

import ctypes

_P = ctypes.c_void_p
_I64 = ctypes.c_int64
KV_BF16, KV_F16 = 0, 1


class KVDesc(ctypes.Structure):
    _fields_ = [("struct_size", ctypes.c_uint32), ("device", ctypes.c_int32), ("dtype", ctypes.c_int32),
                ("num_layers", ctypes.c_int32), ("kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32),
                ("group_size", ctypes.c_int32), ("page_size", ctypes.c_int32), ("num_pages", _I64),
                ("pages", _P), ("bounds", _P), ("reserved", _I64 * 2)]


def declare(L):
    """Argument types of the library's moe_kv_* functions."""
    i32 = ctypes.c_int
    L.moe_kv_sizes.argtypes = [ctypes.POINTER(KVDesc), ctypes.POINTER(_I64), ctypes.POINTER(_I64)]
    L.moe_kv_create.argtypes = [ctypes.POINTER(KVDesc), ctypes.POINTER(_P)]
    L.moe_kv_destroy.argtypes = [_P]
    L.moe_kv_append.argtypes = [_P, i32, _P, _P, _P, _P]
    L.moe_kv_read.argtypes = [_P, i32, _P, _P, _P, _P]
    L.moe_kv_attention.argtypes = [_P, i32, _P, _P, i32, ctypes.c_float, i32, _P, _P, _P, i32, _P]
    L.moe_kv_select.argtypes = [_P, i32, _P, _P, i32, i32, i32, i32, _P, _P]
    L.moe_kv_status.argtypes = [_P]
    L.moe_kv_debug_fail_next_attention.argtypes = [_P]
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


class Handle:
    """What the key/value caches share: self._h, the library's handle, self._c, the binding's
    object over it, and self._destroy, which frees a handle that has none."""

    _h = _c = None

    def close(self):
        """Frees the handle.  MoeError with MOE_ERR_STATE: a call of another thread is running, and the
        cache stays as it is; with MOE_ERR_TIMEOUT: see `check`, and the cache is closed."""
        from . import MoeError
        try:
            if self._c is not None:
                self._c.close()
            elif self._h:
                self._destroy(self._h)
        except MoeError as e:
            if e.status == 5:  # MOE_ERR_STATE
                raise
            self._h = None
            raise
        self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def check(self):
        """Raises MoeError (MOE_ERR_TIMEOUT) where a bounded wait on the device gave up, in a call
        or in a replayed graph that holds one; after a synchronisation."""
        self._c.check()

    def debug_fail_next_attention(self):
        """Test hook: a wait of the next attention runs out (see moe.h)."""
        self._c.debug_fail_next_attention()

    def append(self, k, v, *, table, lens, starts=None, max_new=None, layer=0, stream=None):
        """Quantise the rows k, v into the sequences' pages, and update the pages' bounds (KVCache) or set the
        rows' mass to 0 (KVCache8) where the cache has them."""
        self._c.append(k, v, table, lens, starts, max_new, layer, stream)

    def read(self, k, v, *, table, lens, starts=None, max_new=None, layer=0, stream=None):
        """The stored keys and values of the rows, into k and v."""
        self._c.read(k, v, table, lens, starts, max_new, layer, stream)


class KVCache(Handle):
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
              the most rows of any sequence (None: all rows; which kernel takes the call and how
              it is cut goes by max_new, so it is worth giving).
    These are CUDA tensors and are read on the device only.  Row tensors may be strided
    (16-byte aligned rows and heads, contiguous channels).  Work goes to `stream` (None:
    torch's current stream); where that is not the stream that torch allocated a tensor for, keeping
    the tensor until the work is done is the caller's (Tensor.record_stream)."""

    def __init__(self, pages, *, page_size, head_dim, group_size=64, dtype=None, bounds=None):
        import torch
        from . import MoeError, _kv_binding
        self._lib = _lib()
        self._destroy = self._lib.moe_kv_destroy
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
        self._c = _kv_binding.Cache(MoeError, h.value, d.device, dtype == torch.bfloat16, kv_heads, head_dim)

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

    # The tensors are checked and unpacked in csrc/kv_binding.cpp.

    def attention(self, q, out, *, table, lens, starts=None, max_new=None, scale=None, causal=True, lse=None,
                  pages=None, layer=0, stream=None):
        """out = softmax(scale q k^T) v of the rows q (scale None: 1 / sqrt(head_dim)).
        pages: None, or `select`'s choice, the only pages then attended to.  lse: None, or
        float32 [rows, heads] for the logarithm of each row's sum of exponentials."""
        self._c.attention(q, out, table, lens, starts, max_new, layer, stream, scale, causal, lse, pages)

    def select(self, q, pages, *, table, lens, starts=None, max_new=None, keep_first=1, keep_last=1, layer=0,
               stream=None):
        """Choose pages.shape[-1] pages for each row and kv head into pages (int32 [rows,
        kv_heads, budget], ascending, -1 where a row sees fewer): the first keep_first, the
        last keep_last, then those whose bounds promise the largest q . k."""
        self._c.select(q, pages, table, lens, starts, max_new, layer, stream, keep_first, keep_last)
