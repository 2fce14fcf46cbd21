"""Order, errors, refusals and handles of the 8-bit key/value cache's C entry points, on the host: csrc/kv8.cu
against a runtime of the host's (fake_cuda.cpp) and launchers without kernels."""
import ctypes
import os
import subprocess

import pytest

from conftest import ROOT
from kv_host import Batch, Tensor

P = ctypes.c_void_p


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    from moe_expert_layer_sorted_gb300 import _build as b
    folder = str(tmp_path_factory.mktemp("kv8_host"))
    out = os.path.join(folder, "libkv8_host.so")
    srcs = [os.path.join(b.CSRC, "kv8.cu"), os.path.join(ROOT, "tests", "fake_kernels8.cu"), os.path.join(ROOT, "tests", "fake_cuda.cpp")]
    objs = [os.path.join(folder, os.path.basename(s) + ".o") for s in srcs]
    nvcc = b._nvcc()
    cuda = os.path.join(os.path.dirname(os.path.dirname(nvcc)), "include")
    jobs = [subprocess.Popen([*([nvcc, *b.ARCH, "-Xcompiler"] if s.endswith(".cu") else ["g++", "-I", cuda]), "-fPIC", "-O1",
                              "-std=c++17", "-I", b.INCLUDE, "-I", b.CSRC, "-c", s, "-o", o]) for s, o in zip(srcs, objs)]
    assert not any([j.wait() for j in jobs])
    subprocess.run(["g++", "-shared", "-Wl,-Bsymbolic", "-o", out, *objs, "-lpthread"], check=True)
    L = ctypes.CDLL(out)
    L.fake_log.restype = L.moe_kv8_last_error.restype = ctypes.c_char_p
    L.moe_kv8_last_error.argtypes = [P]
    L.fake_identity.argtypes = [ctypes.c_int, ctypes.c_ulonglong]
    return L


class Cache:
    """A handle over nothing: 2 kv heads, 4 pages."""

    def __init__(self, L, mass=4096):
        from moe_expert_layer_sorted_gb300 import kv8
        self.L, self.h = L, P()
        d = kv8.KV8Desc(struct_size=ctypes.sizeof(kv8.KV8Desc), num_layers=2, kv_heads=2, head_dim=64, page_size=16, num_pages=4,
                        pages=4096, mass=mass)
        assert L.moe_kv8_create(ctypes.byref(d), ctypes.byref(self.h)) == 0
        self.t, self.o = Tensor(4096, 64, 64, 64), Tensor(8192, 64, 64, 64)
        L.fake_clear()

    def batch(self, **kw):
        b = Batch(ctypes.sizeof(Batch), 1, 1, 4, 4, 1, 4096, 4096, None)
        for k, v in kw.items():
            setattr(b, k, v)
        return b

    def append(self, stream=0, layer=0, **kw):
        return self.L.moe_kv8_append(self.h, layer, ctypes.byref(self.batch(**kw)), ctypes.byref(self.t), ctypes.byref(self.o), P(stream))

    def read(self, stream=0, layer=0, **kw):
        return self.L.moe_kv8_read(self.h, layer, ctypes.byref(self.batch(**kw)), ctypes.byref(self.t), ctypes.byref(self.o), P(stream))

    def attention(self, stream=0, layer=0, heads=2, scale=1.0, causal=1, lse=None, weigh=0, out=None, **kw):
        return self.L.moe_kv8_attention(self.h, layer, ctypes.byref(self.batch(**kw)), ctypes.byref(self.t), heads, ctypes.c_float(scale),
                                        causal, ctypes.byref(out or self.o), P(lse), weigh, P(stream))

    def evict(self, stream=0, layer=0, budget=8, first=0, last=0, kept=4096, **kw):
        return self.L.moe_kv8_evict(self.h, layer, ctypes.byref(self.batch(**kw)), budget, first, last, P(kept), P(stream))

    def log(self):
        text = self.L.fake_log().decode().split("\n")[:-1]
        self.L.fake_clear()
        return text


@pytest.fixture
def cache(lib):
    for i in range(16):
        lib.fake_identity(i, 100 + i)
        lib.fake_capturing(i, 0)
    c = Cache(lib)
    yield c
    lib.moe_kv8_destroy(c.h)


def test_another_stream_waits_where_the_workspace_is_used(cache):
    assert cache.attention(4) == 0 and cache.attention(4, lse=4096, weigh=1) == 0
    assert not [x for x in cache.log() if x.startswith("wait")]
    assert cache.attention(5, lse=4096, weigh=1) == 0
    log = cache.log()
    assert log.index("wait 5") < log.index("weigh 5") < log.index("record 5")
    assert cache.append(4) == 0 and cache.read(4) == 0 and cache.evict(4) == 0  # these use none of it
    assert cache.log() == ["append+mass 4", "read 4", "evict 4"]


def test_a_capture_neither_waits_nor_records(cache, lib):
    assert cache.attention(4) == 0
    lib.fake_capturing(5, 1)
    cache.log()
    assert cache.attention(5, lse=4096, weigh=1) == 0
    assert cache.log() == ["weigh 5"]


@pytest.mark.parametrize("call", ["append", "read", "attention", "evict", "status"])
def test_a_wait_that_gave_up_is_reported_once_by_whichever_call_is_next(cache, lib, call):
    def run():
        return lib.moe_kv8_status(cache.h) if call == "status" else getattr(cache, call)(4)

    assert run() == 0
    cache.log()
    lib.fake_raise(cache.h)
    assert run() == 4 and b"gave up" in lib.moe_kv8_last_error(cache.h)
    assert cache.log() == []
    assert run() == 0


def test_the_hook_is_for_one_attention(cache, lib):
    assert lib.moe_kv8_debug_fail_next_attention(cache.h) == 0
    assert cache.attention(4) == 0 and cache.attention(4) == 0
    assert [x for x in cache.log() if "attention" in x] == ["attention that fails 4", "attention 4"]


def test_refusals(cache, lib):
    plain = Cache(lib, mass=None)
    bad = [lambda: cache.attention(lse=None, weigh=1), lambda: cache.attention(lse=4096, weigh=2), lambda: plain.attention(lse=4096, weigh=1),
           lambda: cache.attention(heads=3), lambda: cache.attention(heads=0), lambda: cache.attention(scale=float("inf")),
           lambda: cache.attention(scale=float("nan")), lambda: cache.attention(causal=2), lambda: cache.attention(layer=2),
           lambda: cache.attention(out=cache.t), lambda: cache.attention(out=Tensor(8200, 64, 64, 64)),
           lambda: cache.attention(out=Tensor(8192, 64, 60, 64)), lambda: cache.attention(rows=2), lambda: cache.attention(lens=None),
           lambda: cache.append(layer=-1), lambda: cache.append(table=None), lambda: cache.append(struct_size=3),
           lambda: cache.append(table_stride=3), lambda: cache.append(table_pages=0), lambda: cache.read(batch=-1, rows=-1),
           lambda: cache.evict(budget=0), lambda: cache.evict(first=5, last=4), lambda: cache.evict(first=-1), lambda: cache.evict(last=-1),
           lambda: cache.evict(kept=None), lambda: cache.evict(layer=2), lambda: plain.evict(), lambda: cache.evict(lens=None),
           lambda: cache.evict(first=0x7fffffff, last=0x7fffffff, budget=8)]
    cache.log()
    for i, f in enumerate(bad):
        assert f() == 1, i
    assert cache.evict(budget=0x7fffffff) == 6
    assert cache.log() == []
    # nothing to do is no error
    assert cache.append(batch=0, rows=0) == 0 and cache.attention(max_new=0, rows=0) == 0 and cache.evict(batch=0, rows=0, max_new=0) == 0
    assert cache.log() == []
    assert plain.append(4) == 0 and cache.log() == ["append 4"]
    lib.moe_kv8_destroy(plain.h)


def test_destroy_waits_and_reports(lib):
    c = Cache(lib)
    assert c.attention(4) == 0
    lib.fake_raise(c.h)
    c.log()
    assert lib.moe_kv8_destroy(c.h) == 4 and b"gone" in lib.moe_kv8_last_error(None)
    log = c.log()
    assert log.index("synchronize") < log.index("free")
