"""The key/value cache's C entry points (csrc/kv.cu) built against a runtime of the host's
(fake_cuda.cpp): the order of calls, errors and handles without a GPU."""
import ctypes
import os
import subprocess

from conftest import ROOT

I64, P = ctypes.c_int64, ctypes.c_void_p


class Batch(ctypes.Structure):
    _fields_ = [("struct_size", ctypes.c_uint32), ("batch", ctypes.c_int32), ("max_new", ctypes.c_int32),
                ("table_pages", ctypes.c_int32), ("table_stride", I64), ("rows", I64), ("table", P), ("lens", P), ("starts", P)]


class Tensor(ctypes.Structure):
    _fields_ = [("data", P), ("batch_stride", I64), ("row_stride", I64), ("head_stride", I64)]


def build(folder):
    from moe_expert_layer_sorted_gb300 import _build as b
    lib = os.path.join(str(folder), "libkv_host.so")
    srcs = [os.path.join(b.CSRC, "kv.cu"), os.path.join(ROOT, "tests", "fake_kernels.cu"), os.path.join(ROOT, "tests", "fake_cuda.cpp")]
    objs = [os.path.join(str(folder), os.path.basename(s) + ".o") for s in srcs]
    nvcc = b._nvcc()
    cuda = os.path.join(os.path.dirname(os.path.dirname(nvcc)), "include")
    jobs = [subprocess.Popen([*([nvcc, *b.ARCH, "-Xcompiler"] if s.endswith(".cu") else ["g++", "-I", cuda]), "-fPIC", "-O1",
                              "-std=c++17", "-I", b.INCLUDE, "-I", b.CSRC, "-c", s, "-o", o]) for s, o in zip(srcs, objs)]
    assert not any([j.wait() for j in jobs])
    subprocess.run(["g++", "-shared", "-Wl,-Bsymbolic", "-o", lib, *objs, "-lpthread"], check=True)
    L = ctypes.CDLL(lib)
    L.fake_log.restype = L.moe_kv_last_error.restype = ctypes.c_char_p
    L.moe_kv_last_error.argtypes = [P]
    L.fake_identity.argtypes = [ctypes.c_int, ctypes.c_ulonglong]
    return L


def folder_of(L):
    return os.path.dirname(L._name)


def build_binding(folder):
    """The Python binding over that library: a module."""
    import importlib.util

    from moe_expert_layer_sorted_gb300 import _build as b
    out = os.path.join(str(folder), "_kv_binding.so")
    subprocess.run(b._binding_cmd(out, os.path.join(str(folder), "libkv_host.so")), check=True)
    spec = importlib.util.spec_from_file_location("_kv_binding", out)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


class Cache:
    """A handle over nothing: 1 kv head, 4 pages."""

    def __init__(self, L):
        from moe_expert_layer_sorted_gb300 import kv
        self.L, self.h = L, P()
        d = kv.KVDesc(struct_size=ctypes.sizeof(kv.KVDesc), num_layers=1, kv_heads=1, head_dim=64, group_size=64, page_size=16,
                      num_pages=4, pages=4096, bounds=4096)
        assert L.moe_kv_create(ctypes.byref(d), ctypes.byref(self.h)) == 0
        self.t, self.o = Tensor(4096, 64, 64, 64), Tensor(8192, 64, 64, 64)
        L.fake_clear()

    def batch(self, pages=4):
        return Batch(ctypes.sizeof(Batch), 1, 1, pages, pages, 1, 4096, 4096, None)

    def append(self, stream=0):
        return self.L.moe_kv_append(self.h, 0, ctypes.byref(self.batch()), ctypes.byref(self.t), ctypes.byref(self.o), P(stream))

    def read(self, stream=0):
        return self.L.moe_kv_read(self.h, 0, ctypes.byref(self.batch()), ctypes.byref(self.t), ctypes.byref(self.o), P(stream))

    def attention(self, stream=0):
        return self.L.moe_kv_attention(self.h, 0, ctypes.byref(self.batch()), ctypes.byref(self.t), 1, ctypes.c_float(1.0), 1,
                                       ctypes.byref(self.o), None, None, 0, P(stream))

    def select(self, stream=0, pages=4):
        return self.L.moe_kv_select(self.h, 0, ctypes.byref(self.batch(pages)), ctypes.byref(self.t), 1, 2, 1, 1, P(4096), P(stream))

    def log(self):
        text = self.L.fake_log().decode().split("\n")[:-1]
        self.L.fake_clear()
        return text
