"""The 8-bit key/value cache (see moe_kv8_* in include/moe.h): the handle and its
tensors; the work is done in the CUDA library."""
from __future__ import annotations

import ctypes

from .kv import _I64, _P, KV_BF16, KV_F16, Handle, _bad, _lib


class KV8Desc(ctypes.Structure):
    _fields_ = [("struct_size", ctypes.c_uint32), ("device", ctypes.c_int32), ("dtype", ctypes.c_int32),
                ("num_layers", ctypes.c_int32), ("kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32),
                ("page_size", ctypes.c_int32), ("reserved0", ctypes.c_int32), ("num_pages", _I64),
                ("pages", _P), ("mass", _P), ("reserved", _I64 * 2)]


def declare(L):
    """Argument types of the library's moe_kv8_* functions."""
    i32 = ctypes.c_int
    L.moe_kv8_sizes.argtypes = [ctypes.POINTER(KV8Desc), ctypes.POINTER(_I64), ctypes.POINTER(_I64)]
    L.moe_kv8_create.argtypes = [ctypes.POINTER(KV8Desc), ctypes.POINTER(_P)]
    L.moe_kv8_destroy.argtypes = [_P]
    L.moe_kv8_append.argtypes = [_P, i32, _P, _P, _P, _P]
    L.moe_kv8_read.argtypes = [_P, i32, _P, _P, _P, _P]
    L.moe_kv8_attention.argtypes = [_P, i32, _P, _P, i32, ctypes.c_float, i32, _P, _P, i32, _P]
    L.moe_kv8_evict.argtypes = [_P, i32, _P, i32, i32, i32, _P, _P]
    L.moe_kv8_status.argtypes = [_P]
    L.moe_kv8_debug_fail_next_attention.argtypes = [_P]
    L.moe_kv8_last_error.argtypes = [_P]
    L.moe_kv8_last_error.restype = ctypes.c_char_p


class KVCache8(Handle):
    """A paged key/value cache in 8 bits for `num_layers` layers, with what writes it, reads it,
    attends over it, counts the weight that its tokens get and evicts those that got least.

    pages: uint8 CUDA tensor [num_pages, kv_heads, page_size / 16, block bytes], or with a
    leading layer axis; contiguous.  mass: None, or float32 [num_pages, kv_heads, page_size] with
    the same leading axis, which `append` sets to 0 for new tokens, `attention(weigh=True)` adds
    to and `evict` goes by.  `KVCache8.allocate` makes both.

    A batch of sequences is given to each call as to KVCache's: table, lens, and starts and
    max_new for ragged rows; CUDA tensors that are read on the device only.  Row tensors may be
    strided (16-byte aligned rows and heads, contiguous channels).  Work goes to `stream` (None:
    torch's current stream); where that is not the stream that torch allocated a tensor for, keeping
    the tensor until the work is done is the caller's (Tensor.record_stream)."""

    def __init__(self, pages, *, page_size, head_dim, dtype=None, mass=None):
        import torch
        from . import MoeError, _kv_binding
        self._lib = _lib()
        self._destroy = self._lib.moe_kv8_destroy
        dtype = torch.bfloat16 if dtype is None else dtype
        if dtype not in (torch.bfloat16, torch.float16):
            _bad("dtype must be torch.bfloat16 or torch.float16")
        if not (pages.is_cuda and pages.dtype == torch.uint8 and pages.dim() in (4, 5) and pages.is_contiguous()):
            _bad("pages: contiguous uint8 CUDA tensor [layers,] num_pages, kv_heads, blocks, block bytes")
        shape = tuple(pages.shape)
        layers = shape[0] if len(shape) == 5 else 1
        num_pages, kv_heads = shape[-4], shape[-3]
        want = (num_pages, kv_heads) + self._block_shape(head_dim, page_size)
        if shape[-4:] != want:
            _bad(f"pages: trailing shape {shape[-4:]}, expected {want}")
        if mass is not None:
            if not (mass.device == pages.device and mass.dtype == torch.float32 and mass.is_contiguous()
                    and tuple(mass.shape) == shape[:-4] + (num_pages, kv_heads, page_size)):
                _bad("mass: contiguous float32 [layers,] num_pages, kv_heads, page_size on the pages' device")
        d = KV8Desc()
        d.struct_size = ctypes.sizeof(KV8Desc)
        d.dtype = KV_BF16 if dtype == torch.bfloat16 else KV_F16
        d.num_layers, d.kv_heads, d.head_dim = layers, kv_heads, head_dim
        d.page_size, d.num_pages = page_size, num_pages
        d.device = pages.device.index
        d.pages = pages.data_ptr()
        d.mass = None if mass is None else mass.data_ptr()
        h = _P()
        rc = self._lib.moe_kv8_create(ctypes.byref(d), ctypes.byref(h))
        if rc:
            raise MoeError(rc, self._lib.moe_kv8_last_error(None).decode())
        self._h, self.pages, self.mass, self.desc = h, pages, mass, d
        self.dtype, self.device = dtype, pages.device
        self.layers, self.kv_heads, self.head_dim = layers, kv_heads, head_dim
        self.page_size = page_size
        self._c = _kv_binding.Cache8(MoeError, h.value, d.device, dtype == torch.bfloat16, kv_heads, head_dim)

    @staticmethod
    def _block_shape(head_dim, page_size):
        if page_size < 16:
            _bad("page_size must be 16, 32, 64, 128 or 256")
        return page_size // 16, 32 * head_dim + 16

    @classmethod
    def allocate(cls, num_pages, *, kv_heads, head_dim, page_size=64, dtype=None, layers=1, mass=True, device="cuda"):
        """A cache with pages (and mass) of its own."""
        import torch
        shape = (layers, num_pages, kv_heads)
        pages = torch.empty(shape + cls._block_shape(head_dim, page_size), dtype=torch.uint8, device=device)
        mass = torch.zeros(shape + (page_size,), dtype=torch.float32, device=device) if mass else None
        return cls(pages, page_size=page_size, head_dim=head_dim, dtype=dtype, mass=mass)

    def attention(self, q, out, *, table, lens, starts=None, max_new=None, scale=None, causal=True, lse=None,
                  weigh=False, layer=0, stream=None):
        """out = softmax(scale q k^T) v of the rows q (scale None: 1 / sqrt(head_dim)).
        lse: None, or float32 [rows, heads] for the logarithm of each row's sum of exponentials.
        weigh: add every token's weights in this call to its mass (needs lse, and pages that no two
        sequences of the call share)."""
        self._c.attention(q, out, table, lens, starts, max_new, layer, stream, scale, causal, lse, weigh)

    def evict(self, kept, *, table, lens, keep_first=0, keep_last=0, layer=0, stream=None):
        """Bring every sequence that holds more than kept.shape[-1] tokens back to that many: the
        first keep_first, the last keep_last, and of the others those of the largest mass, moved
        together in their order.  kept int32 [sequences, kv_heads, budget]: the positions that
        stayed, -1 where a sequence held fewer.  Once all layers are done, the lengths are
        lens.clamp_max(budget)."""
        self._c.evict(kept, table, lens, layer, stream, keep_first, keep_last)
