"""Host-side checks of the 8-bit key/value cache's C entry points (no GPU)."""
import ctypes

from test_abi import _lib


def _desc(m, **kw):
    d = m.kv8.KV8Desc()
    d.struct_size = ctypes.sizeof(m.kv8.KV8Desc)
    for k, v in dict(dict(num_layers=2, kv_heads=8, head_dim=128, page_size=64, num_pages=10), **kw).items():
        setattr(d, k, v)
    return d


def test_sizes():
    m = _lib()
    L = m.lib()
    pages, mass = ctypes.c_int64(), ctypes.c_int64()
    for D, P in ((128, 64), (128, 16), (64, 256), (64, 32)):
        d = _desc(m, head_dim=D, page_size=P)
        assert L.moe_kv8_sizes(ctypes.byref(d), ctypes.byref(pages), ctypes.byref(mass)) == 0
        assert pages.value == 10 * 8 * (P // 16) * (32 * D + 16)  # a byte twice per channel, 16 bytes of steps and marks
        assert mass.value == 10 * 8 * P * 4


def test_bad_descriptors_and_null_handles():
    m = _lib()
    L = m.lib()
    n = ctypes.c_int64()
    for bad in (dict(struct_size=8), dict(dtype=2), dict(num_layers=0), dict(kv_heads=0), dict(kv_heads=1025), dict(head_dim=96),
                dict(head_dim=256), dict(page_size=8), dict(page_size=48), dict(page_size=512), dict(num_pages=0),
                dict(num_pages=1 << 31), dict(reserved0=1)):
        d = _desc(m, **bad)
        assert L.moe_kv8_sizes(ctypes.byref(d), ctypes.byref(n), None) == 1, bad
        assert L.moe_kv8_last_error(None)
    d = _desc(m)
    d.reserved[1] = 1
    assert L.moe_kv8_sizes(ctypes.byref(d), ctypes.byref(n), None) == 1
    h = ctypes.c_void_p()
    assert L.moe_kv8_create(None, ctypes.byref(h)) == 1
    assert L.moe_kv8_create(ctypes.byref(_desc(m)), None) == 1
    assert L.moe_kv8_create(ctypes.byref(_desc(m)), ctypes.byref(h)) == 1 and b"pages" in L.moe_kv8_last_error(None)
    assert L.moe_kv8_create(ctypes.byref(_desc(m, pages=24)), ctypes.byref(h)) == 1 and b"aligned" in L.moe_kv8_last_error(None)
    assert L.moe_kv8_create(ctypes.byref(_desc(m, pages=32, mass=8)), ctypes.byref(h)) == 1 and b"aligned" in L.moe_kv8_last_error(None)
    assert not h.value
    assert L.moe_kv8_destroy(None) == 1
    assert L.moe_kv8_status(None) == 1
    assert L.moe_kv8_debug_fail_next_attention(None) == 1
    assert L.moe_kv8_append(None, 0, None, None, None, None) == 1
    assert L.moe_kv8_read(None, 0, None, None, None, None) == 1
    assert L.moe_kv8_attention(None, 0, None, None, 1, 1.0, 1, None, None, 0, None) == 1
    assert L.moe_kv8_evict(None, 0, None, 1, 0, 0, None, None) == 1
