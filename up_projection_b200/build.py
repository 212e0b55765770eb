"""Build libswiglu_b200.so in-tree with nvcc for sm_100a.

    python -m up_projection_b200.build [--force] [--verbose]

Each ``csrc/*.cu`` is compiled to an object under ``_build/`` (in parallel),
then linked into ``up_projection_b200/libswiglu_b200.so`` with the CUDA
runtime linked statically, so the library needs only the driver at run time.
``-Xptxas -v`` output (registers, spills, shared memory per kernel) is kept
in ``_build/ptxas.log``.  ``csrc/binding.cpp``, the native calls of the
operators around the projection, becomes ``_binding<interpreter's suffix>`` next
to it (g++, torch's headers); without it, or with one built for another torch,
those calls go through ctypes.
"""
from __future__ import annotations

import argparse
import concurrent.futures as cf
import glob
import os
import shutil
import subprocess
import sys
import sysconfig
import warnings

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(ROOT, "_build")
LIB = os.path.join(PKG, "libswiglu_b200.so")
BINDING = os.path.join(PKG, "_binding" + sysconfig.get_config_var("EXT_SUFFIX"))

ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
NVCC_FLAGS = ARCH + ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC",
                     "-Xcompiler", "-fvisibility=hidden", "--expt-relaxed-constexpr",
                     "-Xptxas", "-v", f"-I{INCLUDE}", f"-I{CSRC}"]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def _sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _deps_mtime():
    files = _sources() + glob.glob(os.path.join(CSRC, "*.cuh")) + \
        glob.glob(os.path.join(INCLUDE, "*.h")) + [os.path.abspath(__file__)]
    return max(os.path.getmtime(f) for f in files)


def up_to_date() -> bool:
    return os.path.exists(LIB) and os.path.getmtime(LIB) >= _deps_mtime()


def binding_stamp() -> str:
    """What a binding is built for: this torch, its C++ ABI and this interpreter."""
    import torch
    return (f"torch {torch.__version__} abi {int(torch._C._GLIBCXX_USE_CXX11_ABI)} "
            f"python {sysconfig.get_config_var('SOABI')}")


def _stamp_file() -> str:
    return os.path.join(BUILD, "binding.stamp")


def binding_up_to_date() -> bool:
    deps = [os.path.join(CSRC, "binding.cpp"), os.path.join(INCLUDE, "swiglu.h"), os.path.abspath(__file__)]
    if not os.path.exists(BINDING) or os.path.getmtime(BINDING) < max(os.path.getmtime(f) for f in deps):
        return False
    try:
        with open(_stamp_file()) as f:
            return f.read() == binding_stamp()
    except OSError:
        return False


def build_binding(force: bool = False) -> str:
    """Compile csrc/binding.cpp against this interpreter and its torch."""
    if not force and binding_up_to_date():
        return BINDING
    # nothing built for another interpreter or torch is left to be imported
    for old in glob.glob(os.path.join(os.path.dirname(BINDING), "_binding*.so")):
        os.remove(old)
    import torch
    base = os.path.dirname(torch.__file__)
    cuda = os.path.dirname(os.path.dirname(nvcc()))
    tmp = BINDING + f".tmp{os.getpid()}"
    stamp = binding_stamp()
    cmd = [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", f'-DSWIGLU_BUILT_FOR="{stamp}"',
           f"-I{INCLUDE}", "-I" + sysconfig.get_paths()["include"], f"-I{base}/include",
           f"-I{base}/include/torch/csrc/api/include", f"-I{cuda}/include",
           os.path.join(CSRC, "binding.cpp"), "-o", tmp, f"-L{base}/lib", "-ltorch_python", "-ltorch",
           "-ltorch_cpu", "-ltorch_cuda", "-lc10", "-lc10_cuda"]
    p = subprocess.run(cmd, capture_output=True, text=True)
    if p.returncode != 0:
        raise RuntimeError("binding failed:\n" + p.stdout + p.stderr)
    os.replace(tmp, BINDING)
    os.makedirs(BUILD, exist_ok=True)
    with open(_stamp_file(), "w") as f:
        f.write(stamp)
    return BINDING


def _compile(src: str):
    obj = os.path.join(BUILD, os.path.basename(src)[:-3] + ".o")
    cmd = [nvcc(), *NVCC_FLAGS, "-c", src, "-o", obj]
    p = subprocess.run(cmd, capture_output=True, text=True)
    return src, obj, p.returncode, p.stdout + p.stderr


def build(force: bool = False, verbose: bool = False) -> str:
    """The library, then the binding, whose failure is a warning."""
    if force or not up_to_date():
        _build_library(verbose)
    try:
        build_binding(force)
    except Exception as e:  # no compiler, no headers, a torch it does not fit
        warnings.warn(f"no native binding, its calls go through ctypes: {e}")
    return LIB


def _build_library(verbose: bool):
    os.makedirs(BUILD, exist_ok=True)
    srcs = _sources()
    logs = []
    with cf.ThreadPoolExecutor(max_workers=min(8, len(srcs))) as ex:
        results = list(ex.map(_compile, srcs))
    failed = False
    for src, _obj, rc, out in results:
        logs.append(f"=== {os.path.basename(src)} (rc={rc})\n{out}")
        if rc != 0:
            failed = True
    with open(os.path.join(BUILD, "ptxas.log"), "w") as f:
        f.write("\n".join(logs))
    if failed:
        raise RuntimeError("nvcc failed:\n" + "\n".join(l for l in logs if "rc=0" not in l))
    if verbose:
        print("\n".join(logs))
    tmp = LIB + f".tmp{os.getpid()}"
    cmd = [nvcc(), *ARCH, "-shared", "-cudart", "static", "-o", tmp,
           *[r[1] for r in results], "-lpthread", "-ldl", "-lrt"]
    p = subprocess.run(cmd, capture_output=True, text=True)
    if p.returncode != 0:
        raise RuntimeError("link failed:\n" + p.stdout + p.stderr)
    os.replace(tmp, LIB)


def main(argv=None):
    ap = argparse.ArgumentParser()
    ap.add_argument("--force", action="store_true")
    ap.add_argument("--verbose", action="store_true")
    a = ap.parse_args(argv)
    print(build(force=a.force, verbose=a.verbose))


if __name__ == "__main__":
    sys.exit(main())
