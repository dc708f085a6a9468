"""Build ``libgdn2.so`` (the C-ABI CUDA library) in-tree with nvcc for sm_103a.

Each ``csrc/*.cu`` is compiled to an object in parallel, then linked into
``gated_deltanet_prefill_gb300/_build/libgdn2.so``.  The build is skipped when
the library is newer than every source and header.  ``csrc/gdn2_attn_call.cpp``
(a CPython module that calls the library for ``attn.py``) is compiled beside
them with the host compiler; where that fails, the library is linked all the
same, for the C ABI and ``gdn2.py``, before the error is raised.
"""
from __future__ import annotations

import glob
import os
import shutil
import subprocess
import sysconfig
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(BUILD, "libgdn2.so")
# the checked build: the same sources with the device-side index checks on
# (-DGDN2_CHECK_BOUNDS); built on request only (tests), never the product path
LIB_CHECKED = os.path.join(BUILD, "libgdn2_checked.so")
CALL_SOURCE = os.path.join(CSRC, "gdn2_attn_call.cpp")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC,-fvisibility=hidden", "--expt-relaxed-constexpr",
         "-I", INCLUDE, "-I", CSRC]


def nvcc() -> str:
    home = os.environ.get("CUDA_HOME", "/usr/local/cuda")
    cand = os.path.join(home, "bin", "nvcc")
    return cand if os.path.exists(cand) else (shutil.which("nvcc") or "nvcc")


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _stale(lib=LIB) -> bool:
    if not os.path.exists(lib):
        return True
    t = os.path.getmtime(lib)
    deps = sources() + [f for d, x in ((CSRC, "*.cuh"), (CSRC, "*.h"), (INCLUDE, "*.h"))
                        for f in glob.glob(os.path.join(d, x))]
    return any(os.path.getmtime(f) > t for f in deps)


def call_path() -> str:
    """The calls module for this Python and this torch, whose internals it is compiled against."""
    import torch
    return os.path.join(BUILD, "gdn2_attn_call.%s-torch%s.so" % (sysconfig.get_config_var("SOABI"), torch.__version__))


def _call_stale() -> bool:
    call = call_path()
    if not os.path.exists(call):
        return True
    t = os.path.getmtime(call)
    return any(os.path.getmtime(f) > t for f in [CALL_SOURCE] + glob.glob(os.path.join(INCLUDE, "*.h")))


def _build_call() -> None:
    import torch  # its headers and libraries: the module takes and returns torch's tensors
    home = os.path.dirname(os.path.abspath(torch.__file__))
    lib = os.path.join(home, "lib")
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(nvcc())))
    os.makedirs(BUILD, exist_ok=True)
    call = call_path()
    tmp = call + ".%d.tmp" % os.getpid()
    cmd = ["g++", "-std=c++17", "-O2", "-fPIC", "-fvisibility=hidden", "-shared", CALL_SOURCE, "-o", tmp,
           "-D_GLIBCXX_USE_CXX11_ABI=%d" % torch._C._GLIBCXX_USE_CXX11_ABI, "-I", INCLUDE]
    for d in (os.path.join(home, "include"), os.path.join(home, "include", "torch", "csrc", "api", "include"),
              os.path.join(cuda, "include"), sysconfig.get_paths()["include"]):
        cmd += ["-isystem", d]
    cmd += ["-L" + lib, "-Wl,-rpath," + lib] + ["-l" + x for x in ("c10", "c10_cuda", "torch_cpu", "torch_cuda", "torch_python")]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        print(" ".join(cmd))
        print(r.stdout + r.stderr)
        raise RuntimeError("g++ failed on %s" % CALL_SOURCE)
    os.replace(tmp, call)


def build(force: bool = False, verbose: bool = False, extra_flags=(), checked: bool = False) -> str:
    """Build libgdn2.so (or, with checked=True, libgdn2_checked.so: the
    device-side index checks compiled in) and return its path."""
    lib = LIB_CHECKED if checked else LIB
    call = not checked and (force or _call_stale())
    if not force and not _stale(lib):
        if call:
            _build_call()
        return lib
    odir = os.path.join(BUILD, "checked") if checked else BUILD
    os.makedirs(odir, exist_ok=True)
    if checked:
        extra_flags = tuple(extra_flags) + ("-DGDN2_CHECK_BOUNDS",)
    srcs = sources()
    objs = [os.path.join(odir, os.path.basename(s)[:-3] + ".o") for s in srcs]

    def compile_one(pair):
        src, obj = pair
        cmd = [nvcc(), "-c", src, "-o", obj] + ARCH + FLAGS + list(extra_flags)
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0 or verbose:
            print(" ".join(cmd))
            print(r.stdout + r.stderr)
        if r.returncode != 0:
            raise RuntimeError("nvcc failed on %s" % src)

    with ThreadPoolExecutor(max_workers=max(1, min(len(srcs) + 1, os.cpu_count() or 1))) as ex:
        module = ex.submit(_build_call) if call else None
        list(ex.map(compile_one, zip(srcs, objs)))
    tmp = lib + ".%d.tmp" % os.getpid()
    cmd = [nvcc(), "-shared", "-o", tmp] + objs + ARCH
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        print(" ".join(cmd)); print(r.stdout + r.stderr)
        raise RuntimeError("link failed")
    os.replace(tmp, lib)
    if module:
        module.result()  # (the library is there whether or not the module could be built)
    return lib


if __name__ == "__main__":
    print(build(force=True, verbose=True))
