"""Builds ``libmimo_attn.so`` in-tree with nvcc for sm_100a, and the native part of
the Python binding (``_fast_call``) with the host compiler."""

from __future__ import annotations

import os
import subprocess

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
SRC = os.path.join(PKG, "csrc", "mimo_attn.cu")
LIB = os.path.join(PKG, "libmimo_attn.so")
# the same sources with every kernel's row indices bounds-checked (-DMIMO_CHECKED)
LIB_CHECKED = os.path.join(PKG, "libmimo_attn_checked.so")
DEPS = [
    os.path.join(PKG, "csrc", f)
    for f in ("mimo_attn.cu", "common.cuh", "decode_kernel.cuh", "prefill_kernel.cuh",
              "prefill_swa_kernel.cuh", "decode_fp8_kernel.cuh",
              "rope_append_kernel.cuh", "decode_merge_kernel.cuh",
              "paged_common.cuh", "paged_attention_kernel.cuh", "paged_window_kernel.cuh", "paged_decode_kernel.cuh",
              "paged_append_kernel.cuh",
              "page_table_kernel.cuh", "page_copy_kernel.cuh",
              "backward_kernel.cuh", "backward_tc_kernel.cuh", "backward_dq_tc_kernel.cuh")
] + [os.path.join(ROOT, "include", "mimo_attn.h")]

NVCC_FLAGS = [
    "-O3", "-std=c++17",
    "-gencode", "arch=compute_100a,code=sm_100a",
    "-lineinfo",
    "-Xcompiler", "-fPIC", "-shared", "-cudart", "static",
]


def nvcc_path():
    for cand in (os.environ.get("NVCC"), "/usr/local/cuda/bin/nvcc", "nvcc"):
        if cand and (os.path.sep not in cand or os.path.exists(cand)):
            return cand
    return "nvcc"


def up_to_date(lib=LIB):
    if not os.path.exists(lib):
        return False
    t = os.path.getmtime(lib)
    return all(os.path.getmtime(d) <= t for d in DEPS if os.path.exists(d))


def build(force=False, verbose=False, checked=False):
    """Compile the library (or, with checked=True, its bounds-checked variant) if
    any source is newer than it; returns the .so path."""
    lib = LIB_CHECKED if checked else LIB
    if not force and up_to_date(lib):
        return lib
    extra = ["-DMIMO_CHECKED"] if checked else []
    cmd = [nvcc_path(), *NVCC_FLAGS, *extra, "-Xptxas", "-v", "-o", lib, SRC]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError("nvcc failed:\n" + res.stdout + res.stderr)
    if verbose:
        print(res.stderr)
    return lib


FAST_SRC = os.path.join(PKG, "csrc", "fast_call.cpp")


def fast_call_path():
    import sysconfig

    return os.path.join(PKG, "_fast_call" + sysconfig.get_config_var("EXT_SUFFIX"))


def build_fast_call(force=False):
    """Compile the binding's native calls against the installed torch if their source is
    newer than them; returns the .so path."""
    import sysconfig

    import torch
    from torch.utils import cpp_extension

    so = fast_call_path()
    deps = (FAST_SRC, os.path.join(ROOT, "include", "mimo_attn.h"))
    if not force and os.path.exists(so) and all(os.path.getmtime(d) <= os.path.getmtime(so) for d in deps):
        return so
    include = [*cpp_extension.include_paths("cuda"), sysconfig.get_paths()["include"]]
    libs = cpp_extension.library_paths("cuda")
    cmd = [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-shared",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           *(f"-I{d}" for d in include), FAST_SRC, "-o", so, *(f"-L{d}" for d in libs),
           "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_cuda", "-ltorch_python"]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError("the binding's native calls failed to compile:\n" + res.stdout + res.stderr)
    return so


if __name__ == "__main__":
    import sys

    build(force=True, verbose=True, checked="--checked" in sys.argv)
    build_fast_call()
