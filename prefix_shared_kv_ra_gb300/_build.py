"""Build the CUDA library libra.so in-tree (nvcc, sm_103a only).

Each translation unit is compiled in parallel to an object file under
``_build/``; they are linked into ``prefix_shared_kv_ra_gb300/libra.so``
(static cudart, no libcuda link dependency: the driver entry points the
library needs are resolved at run time).  ``_ra_binding.*.so`` beside it is the Python
side of the small operators, C++ on torch's tensors: it fits the Python and torch it was built
with only, which its name gives.  A rebuild happens only when a
source or header is newer than the library.
"""
from __future__ import annotations

import concurrent.futures as cf
import glob
import importlib.util
import os
import shutil
import subprocess
import sys
import sysconfig

import torch

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libra.so")
# argument checks of the small operators (CPython API and torch's C++ tensors)
BINDING = os.path.join(PKG, f"_ra_binding.{sysconfig.get_config_var('SOABI')}.torch{torch.__version__}.so")
SOURCES = ["api_common.cu", "kv_store.cu", "decode.cu", "decode_mod.cu", "extend.cu", "extend_mod.cu", "decode_static.cu",
           "kv8_store.cu", "decode_kv8.cu", "qk_norm_rope.cu", "tree.cu", "tree_narrow.cu", "tree_verify.cu",
           "step_slots.cu"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "--expt-relaxed-constexpr",
              "-Xptxas", "-warn-spills"]


def _nvcc() -> str:
    for cand in (os.environ.get("NVCC"), "/usr/local/cuda/bin/nvcc", "nvcc"):
        if cand and (os.path.isabs(cand) and os.path.exists(cand) or not os.path.isabs(cand)):
            return cand
    return "nvcc"


def _deps():
    return (glob.glob(os.path.join(CSRC, "*")) + glob.glob(os.path.join(ROOT, "include", "*.h"))
            + [os.path.abspath(__file__)])


def _stale(target: str) -> bool:
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(d) > t for d in _deps())


def build_binding(force: bool = False) -> str:
    if not force and not _stale(BINDING):
        return BINDING
    torch_dir = importlib.util.find_spec("torch").submodule_search_locations[0]
    torch_lib = os.path.join(torch_dir, "lib")
    cuda_include = os.path.join(os.path.dirname(os.path.dirname(shutil.which(_nvcc()) or _nvcc())), "include")
    tmp = BINDING + f".tmp{os.getpid()}"
    r = subprocess.run([os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-Wall", "-Wno-missing-field-initializers", "-shared",
                        "-fPIC", "-I", sysconfig.get_paths()["include"], "-I", os.path.join(torch_dir, "include"), "-I",
                        cuda_include, os.path.join(CSRC, "py_binding.cpp"), "-o", tmp, "-L", torch_lib, "-ltorch_python",
                        "-ltorch_cpu", "-lc10_cuda", "-lc10", f"-Wl,-rpath,{torch_lib}"], capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed for py_binding.cpp:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, BINDING)
    return BINDING


def build(force: bool = False, verbose: bool = False, ptxas_verbose: bool = False) -> str:
    if not force and not _stale(LIB):
        build_binding()
        return LIB
    os.makedirs(BUILD, exist_ok=True)
    nvcc = _nvcc()
    extra = ["-Xptxas", "-v"] if ptxas_verbose else []

    def compile_one(src: str) -> str:
        obj = os.path.join(BUILD, os.path.splitext(src)[0] + ".o")
        cmd = [nvcc, *ARCH, *NVCC_FLAGS, *extra, "-I", os.path.join(ROOT, "include"), "-c",
               os.path.join(CSRC, src), "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed for {src}:\n{r.stdout}\n{r.stderr}")
        if verbose or ptxas_verbose:
            sys.stderr.write(r.stdout + r.stderr)
        return obj

    with cf.ThreadPoolExecutor(max_workers=len(SOURCES) + 1) as ex:
        binding = ex.submit(build_binding, force)
        objs = list(ex.map(compile_one, SOURCES))
        binding.result()
    tmp = LIB + f".tmp{os.getpid()}"
    r = subprocess.run([nvcc, *ARCH, "-shared", "-o", tmp, *objs], capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose=True, ptxas_verbose="-v" in sys.argv)
    print(LIB)
