"""Host-side checks of the key/value cache's C entry points (no GPU)."""
import ctypes

from test_abi import _lib


def _desc(m, **kw):
    d = m.kv.KVDesc()
    d.struct_size = ctypes.sizeof(m.kv.KVDesc)
    for k, v in dict(dict(num_layers=2, kv_heads=8, head_dim=128, group_size=64, page_size=64, num_pages=10), **kw).items():
        setattr(d, k, v)
    return d


def test_sizes():
    m = _lib()
    L = m.lib()
    pages, bounds = ctypes.c_int64(), ctypes.c_int64()
    for D, G, P in ((128, 64, 64), (128, 32, 16), (64, 64, 256), (128, 128, 32), (64, 32, 128)):
        d = _desc(m, head_dim=D, group_size=G, page_size=P)
        assert L.moe_kv_sizes(ctypes.byref(d), ctypes.byref(pages), ctypes.byref(bounds)) == 0
        assert pages.value == 10 * 8 * P * (D + 8 * (D // G))  # 4 bits twice, two 16-bit params per group twice
        assert bounds.value == 10 * 8 * 2 * D * 2


def test_bad_descriptors_and_null_handles():
    m = _lib()
    L = m.lib()
    n = ctypes.c_int64()
    for bad in (dict(struct_size=8), dict(dtype=2), dict(num_layers=0), dict(kv_heads=0), dict(kv_heads=1025), dict(head_dim=96),
                dict(group_size=16), dict(group_size=256), dict(head_dim=64, group_size=128), dict(page_size=8),
                dict(page_size=48), dict(page_size=512), dict(num_pages=0), dict(num_pages=1 << 31)):
        d = _desc(m, **bad)
        assert L.moe_kv_sizes(ctypes.byref(d), ctypes.byref(n), None) == 1, bad
        assert L.moe_kv_last_error(None)
    h = ctypes.c_void_p()
    assert L.moe_kv_create(None, ctypes.byref(h)) == 1
    assert L.moe_kv_create(ctypes.byref(_desc(m)), None) == 1
    assert L.moe_kv_create(ctypes.byref(_desc(m)), ctypes.byref(h)) == 1 and b"pages" in L.moe_kv_last_error(None)
    assert L.moe_kv_create(ctypes.byref(_desc(m, pages=24)), ctypes.byref(h)) == 1 and b"aligned" in L.moe_kv_last_error(None)
    assert not h.value
    assert L.moe_kv_destroy(None) == 1
    assert L.moe_kv_append(None, 0, None, None, None, None) == 1
    assert L.moe_kv_read(None, 0, None, None, None, None) == 1
    assert L.moe_kv_attention(None, 0, None, None, 1, 1.0, 1, None, None, None, 0, None) == 1
    assert L.moe_kv_select(None, 0, None, None, 1, 1, 0, 1, None, None) == 1
