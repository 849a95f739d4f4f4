"""Build the C-ABI library libfd.so (nvcc, sm_100a) and the Python binding's module in-tree.

Usage: python split_kv_decode_flashdecoding_b200/build.py [--force] [-v]
(run by path: importing the package needs the library already built)

The CUDA runtime is linked statically and the driver entry points the library needs are
fetched at run time, so the library loads on a machine without a GPU driver (its attention
calls then fail with FD_ERR_CUDA) and needs nothing but the driver on a GPU machine. The module
(csrc/binding.cpp) marshals the serving calls' tensors for libfd.so and is linked to torch.
"""

from __future__ import annotations

import argparse
import concurrent.futures as cf
import importlib.util
import os
import re
import shutil
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libfd.so")
BINDING = os.path.join(PKG, "_fd_binding.so")
BINDING_STAMP = os.path.join(BUILD, "_fd_binding.txt")  # what BINDING was built for
BINDING_SRC = os.path.join(CSRC, "binding.cpp")
INCLUDE = os.path.join(ROOT, "include")

ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
NVCC_FLAGS = ARCH + ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC",
                     "-Xcompiler", "-Wall", "--expt-relaxed-constexpr", "-I", INCLUDE, "-I", CSRC]


def nvcc() -> str:
    exe = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(exe):
        raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libfd.so")
    return exe


def sources():
    return sorted(os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith(".cu"))


def _deps():
    deps = sources()
    deps += [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith((".h", ".cuh"))]
    deps.append(os.path.join(INCLUDE, "fd.h"))
    return deps


def _newer(target: str, deps) -> bool:
    return os.path.exists(target) and all(os.path.getmtime(d) <= os.path.getmtime(target) for d in deps)


def up_to_date() -> bool:
    return _newer(LIB, _deps())


def _compile(src: str, verbose: bool) -> str:
    obj = os.path.join(BUILD, os.path.basename(src)[:-3] + ".o")
    cmd = [nvcc(), *NVCC_FLAGS, "-c", src, "-o", obj]
    if verbose:
        cmd += ["-Xptxas", "-v"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc failed for {src}:\n{r.stdout}\n{r.stderr}")
    if verbose:
        sys.stderr.write(r.stderr)
    return obj


def _torch_dir() -> str:
    spec = importlib.util.find_spec("torch")
    if spec is None or not spec.submodule_search_locations:
        raise RuntimeError("torch not found: the binding is built against it")
    return list(spec.submodule_search_locations)[0]


def _torch_version() -> str:
    with open(os.path.join(_torch_dir(), "version.py"), encoding="utf-8") as f:
        return re.search(r"^__version__ = ['\"](.+)['\"]", f.read(), re.M).group(1)


def _binding_is_for() -> str:
    """What the module depends on besides its source: torch's and Python's binary interfaces."""
    return f"torch {_torch_version()} in {_torch_dir()}, python {sysconfig.get_config_var('SOABI')}"


def binding_up_to_date() -> bool:
    if not _newer(BINDING, [BINDING_SRC, os.path.join(INCLUDE, "fd.h")]) or not os.path.exists(BINDING_STAMP):
        return False
    with open(BINDING_STAMP, encoding="utf-8") as f:
        return f.read() == _binding_is_for()


def build_binding(force: bool = False) -> str:
    """Compile csrc/binding.cpp against torch and libfd.so (which has to be there); returns its path."""
    if not force and binding_up_to_date():
        return BINDING
    torch_dir, cuda = _torch_dir(), os.path.dirname(os.path.dirname(os.path.realpath(nvcc())))
    cxx = shutil.which("g++") or "c++"
    tmp = BINDING + ".tmp"
    cmd = [cxx, "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden", "-Wall",
           f'-DFD_TORCH_VERSION="{_torch_version()}"',
           *(x for d in (os.path.join(torch_dir, "include"), sysconfig.get_paths()["include"], os.path.join(cuda, "include"))
             for x in ("-isystem", d)),
           "-I", INCLUDE, BINDING_SRC, "-o", tmp, "-L", PKG, "-l:libfd.so", "-L", os.path.join(torch_dir, "lib"),
           "-ltorch_python", "-ltorch", "-ltorch_cpu", "-lc10", "-lc10_cuda",
           "-l:libstdc++.so.6", "-Wl,-rpath,$ORIGIN"]  # the libstdc++ that torch uses, by name
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"building the binding failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, BINDING)
    os.makedirs(BUILD, exist_ok=True)
    with open(BINDING_STAMP, "w", encoding="utf-8") as f:
        f.write(_binding_is_for())
    return BINDING


def build(force: bool = False, verbose: bool = False) -> str:
    """Compile every .cu under csrc/, link libfd.so and build the binding's module; returns
    libfd.so's path."""
    if not force and up_to_date():
        build_binding()
        return LIB
    os.makedirs(BUILD, exist_ok=True)
    srcs = sources()
    with cf.ThreadPoolExecutor(max_workers=min(8, len(srcs))) as ex:
        objs = list(ex.map(lambda s: _compile(s, verbose), srcs))
    tmp = LIB + ".tmp"
    cmd = [nvcc(), *ARCH, "--shared", "-Xcompiler", "-fPIC", "-o", tmp, *objs]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)
    build_binding(force)
    return LIB


def main():
    ap = argparse.ArgumentParser()
    ap.add_argument("--force", action="store_true")
    ap.add_argument("-v", "--verbose", action="store_true", help="print ptxas resource usage")
    a = ap.parse_args()
    print(build(force=a.force, verbose=a.verbose))


if __name__ == "__main__":
    main()
