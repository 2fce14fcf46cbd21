"""Build of the CUDA library (sm_103a only): one nvcc per translation unit, in
parallel, then one shared-library link, and of the key/value cache's Python
binding where torch is installed.  Output: libmoe_gb300.so and _kv_binding.so in
moe_expert_layer_sorted_gb300/ (git-ignored, rebuilt per box)."""
from __future__ import annotations

import concurrent.futures as cf
import importlib.metadata
import importlib.util
import os
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(ROOT, "_build")
LIB = os.path.join(PKG, "libmoe_gb300.so")
BINDING = os.path.join(PKG, "_kv_binding.so")
SOURCES = ["plan.cu", "decode.cu", "prefill.cu", "cache.cu", "noalloc.cu", "kv.cu", "kv_append.cu",
           "kv_attention.cu", "kv_select.cu", "kv_decode_bf16.cu", "kv_decode_f16.cu",
           "kv_prompt_bf16.cu", "kv_prompt_f16.cu"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-I", INCLUDE, "-I", CSRC]


def _nvcc() -> str:
    cand = os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "bin", "nvcc")
    return cand if os.path.exists(cand) else "nvcc"


def _deps():
    hdrs = [os.path.join(INCLUDE, "moe.h")] + [os.path.join(CSRC, f) for f in os.listdir(CSRC)
                                                if f.endswith((".h", ".cuh"))]
    return max(os.path.getmtime(h) for h in hdrs)


def _binding_for() -> str | None:
    """What a binding is built for (it holds torch's and the interpreter's layouts); None without torch."""
    spec = importlib.util.find_spec("torch")
    if spec is None:
        return None
    try:
        version = importlib.metadata.version("torch")
    except importlib.metadata.PackageNotFoundError:  # not installed as a package: by its files
        version = f"{spec.origin} of {os.path.getmtime(spec.origin)}"
    return f"torch {version}, python {sys.version}"


def _binding_fresh(made_for: str) -> bool:
    files = [os.path.join(CSRC, "kv_binding.cpp"), os.path.join(INCLUDE, "moe.h")]
    try:
        with open(BINDING + ".for") as f:
            return f.read() == made_for and os.path.getmtime(BINDING) >= max(os.path.getmtime(x) for x in files)
    except OSError:
        return False


def _binding_cmd(out: str, lib: str = LIB) -> list:
    """g++ command of the key/value cache's Python binding over `lib`, into `out`."""
    src = os.path.join(CSRC, "kv_binding.cpp")
    import sysconfig

    import torch
    t = os.path.dirname(torch.__file__)
    cuda = os.path.dirname(os.path.dirname(_nvcc()))
    inc = [INCLUDE, os.path.join(t, "include"), os.path.join(t, "include", "torch", "csrc", "api", "include"),
           os.path.join(cuda, "include"), sysconfig.get_paths()["include"]]
    return ["g++", "-O2", "-std=c++17", "-fPIC", "-shared", f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
            *[f"-I{i}" for i in inc], src, "-o", out, f"-L{os.path.dirname(lib)}", f"-L{os.path.join(t, 'lib')}", f"-l:{os.path.basename(lib)}",
            "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_python", "-Wl,-rpath,$ORIGIN"]


def build(verbose: bool = False, force: bool = False) -> str:
    os.makedirs(BUILD, exist_ok=True)
    nvcc = _nvcc()
    dep_t = _deps()
    srcs = [s for s in SOURCES if os.path.exists(os.path.join(CSRC, s))]
    objs = []
    jobs = []
    for s in srcs:
        src = os.path.join(CSRC, s)
        obj = os.path.join(BUILD, s.replace(".cu", ".o"))
        objs.append(obj)
        if force or not os.path.exists(obj) or os.path.getmtime(obj) < max(os.path.getmtime(src), dep_t):
            jobs.append([nvcc, *ARCH, *FLAGS, "-c", src, "-o", obj])
    if jobs:
        with cf.ThreadPoolExecutor(max_workers=len(jobs)) as ex:
            futs = [ex.submit(subprocess.run, j, capture_output=True, text=True) for j in jobs]
            for j, f in zip(jobs, futs):
                r = f.result()
                if verbose or r.returncode:
                    print(" ".join(j))
                    print(r.stdout + r.stderr)
                if r.returncode:
                    raise RuntimeError(f"nvcc failed for {j[-3]}")
    if jobs or force or not os.path.exists(LIB):
        cuda_lib = os.path.join(os.path.dirname(os.path.dirname(nvcc)), "lib64")
        cmd = [nvcc, *ARCH, "-shared", "-o", LIB + ".tmp", *objs, "-lcublas", "-Xlinker", f"-rpath,{cuda_lib}"]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode:
            print(" ".join(cmd))
            print(r.stdout + r.stderr)
            raise RuntimeError("link failed")
        os.replace(LIB + ".tmp", LIB)
    made_for = _binding_for()  # without torch there is the C library alone
    if made_for and not _binding_fresh(made_for):
        cmd = _binding_cmd(BINDING + ".tmp")
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode:
            print(" ".join(cmd))
            print(r.stdout + r.stderr)
            raise RuntimeError("the Python binding did not build")
        os.replace(BINDING + ".tmp", BINDING)
        with open(BINDING + ".for", "w") as f:
            f.write(made_for)
    return LIB


if __name__ == "__main__":
    print(build(verbose=True))
