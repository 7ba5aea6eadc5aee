"""Build libgqa_attn.so and _cache_ext.so in-tree.

Each .cu translation unit is compiled in parallel with nvcc for sm_103a into
_build/, then linked into causal_gqa_attention_fwd_gb300/libgqa_attn.so with
the CUDA runtime linked statically (the library does not need libcuda at load
time; the driver's tensor-map encoder is fetched at run time).  Beside them g++
compiles the CPython module of the cache operators against the installed
PyTorch's headers.
"""
from __future__ import annotations

import os
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(ROOT, "_build")
LIB = os.path.join(PKG, "libgqa_attn.so")
DEBUG_LIB = os.path.join(PKG, "libgqa_attn_debug.so")
EXT = os.path.join(PKG, "_cache_ext.so")
EXT_SOURCE = os.path.join(CSRC, "cache_binding.cpp")

SOURCES = ["api.cu", "attn_fwd.cu", "attn_bwd.cu", "attn_bwd_split.cu", "attn_decode.cu",
           "cache_api.cu", "cache_ops.cu", "attn_decode_q4.cu", "attn_prefix.cu", "attn_own.cu", "cache_evict.cu"]
HEADERS = ["sm103.cuh", "kernels.h", "tmap.h", "rope.h", "bwd_common.cuh", "api_util.h", "cache_ops.h", "fp4.cuh",
           "stream.cuh", "own_keys.cuh", "share_out.h"]

NVCC_FLAGS = [
    "-gencode", "arch=compute_103a,code=sm_103a",
    "-O3", "-std=c++17", "-lineinfo",
    "-Xcompiler", "-fPIC", "-Xcompiler", "-fvisibility=hidden",
    "-I" + INCLUDE, "-I" + CSRC,
]


def _nvcc():
    cand = os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "bin", "nvcc")
    return cand if os.path.exists(cand) else "nvcc"


def _stale(out, deps):
    if not os.path.exists(out):
        return True
    t = os.path.getmtime(out)
    return any(os.path.getmtime(d) > t for d in deps)


def _ext_command(out):
    """The g++ command that builds the CPython module, and the PyTorch it is for."""
    import torch
    root = os.path.dirname(torch.__file__)
    lib = os.path.join(root, "lib")
    return ["g++", "-O2", "-std=c++17", "-shared", "-fPIC", "-fvisibility=hidden",
            "-D_GLIBCXX_USE_CXX11_ABI=%d" % torch._C._GLIBCXX_USE_CXX11_ABI, "-I" + INCLUDE,
            "-I" + sysconfig.get_paths()["include"], "-isystem", os.path.join(root, "include"), EXT_SOURCE, "-o", out,
            "-L" + lib, "-Wl,-rpath," + lib, "-ltorch_python", "-ltorch_cpu", "-lc10"], torch.__version__


def build(force: bool = False, verbose: bool = False, extra_flags=(), debug: bool = False) -> str:
    """Build the library (debug=True: the -DGQA_DEBUG variant with bounds checks in the kernels,
    libgqa_attn_debug.so, objects in _build/debug)."""
    build_dir = os.path.join(BUILD, "debug") if debug else BUILD
    lib_path = DEBUG_LIB if debug else LIB
    if debug:
        extra_flags = (*extra_flags, "-DGQA_DEBUG")
    os.makedirs(build_dir, exist_ok=True)
    nvcc = _nvcc()
    hdrs = [os.path.join(CSRC, h) for h in HEADERS] + [os.path.join(INCLUDE, "gqa_attn.h")]
    objs, procs = [], []
    for src in SOURCES:
        s = os.path.join(CSRC, src)
        o = os.path.join(build_dir, src.replace(".cu", ".o"))
        objs.append(o)
        if force or _stale(o, [s] + hdrs):
            cmd = [nvcc, *NVCC_FLAGS, *extra_flags, "-c", s, "-o", o]
            if verbose:
                cmd.insert(1, "-Xptxas=-v")
            procs.append((src, subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT)))
    stamp, ext_tmp = os.path.join(BUILD, "cache_ext.torch"), EXT + ".tmp%d" % os.getpid()
    ext_cmd, version = _ext_command(ext_tmp)
    built_for = open(stamp).read() if os.path.exists(stamp) else ""
    ext = force or built_for != version or _stale(EXT, [EXT_SOURCE, os.path.join(INCLUDE, "gqa_attn.h")])
    if ext:
        procs.append(("cache_binding.cpp", subprocess.Popen(ext_cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT)))
    failed = []
    for src, p in procs:
        out, _ = p.communicate()
        if verbose or p.returncode:
            sys.stdout.write(out.decode())
        if p.returncode:
            failed.append(src)
    if failed:
        raise RuntimeError(f"the compiler failed for {failed}")
    if ext:
        os.replace(ext_tmp, EXT)
        with open(stamp, "w") as f:
            f.write(version)
    if force or procs or _stale(lib_path, objs):
        tmp = lib_path + ".tmp%d" % os.getpid()
        cmd = [nvcc, "-shared", "-gencode", "arch=compute_103a,code=sm_103a", "-cudart", "static",
               "-Xcompiler", "-fPIC", *objs, "-o", tmp]
        subprocess.run(cmd, check=True)
        os.replace(tmp, lib_path)
    return lib_path


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose="-v" in sys.argv, debug="--debug" in sys.argv)
