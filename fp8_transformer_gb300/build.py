"""Builds libte_gb300.so in-tree with nvcc for sm_103a.

Each translation unit is compiled in parallel, then linked into one shared library next to this
file.  A second, small library reads torch tensors for the binding; it is built against the headers of
the installed torch and carries its version in its name.  The build is skipped when both are newer than
every source.
"""

from __future__ import annotations

import os
import shutil
import subprocess
import sys
import sysconfig
from concurrent.futures import ThreadPoolExecutor

import torch

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD_DIR = os.path.join(HERE, "_build")
LIB_NAME = "libte_gb300.so"
LIB_PATH = os.path.join(HERE, LIB_NAME)
SOURCES = ["api.cu", "norm.cu", "elementwise.cu", "gemm.cu", "tmap.cu", "profile.cu", "noalloc.cu",
           "selftest.cu", "host_pipeline.cu", "block_quant.cu", "block_gemm.cu", "block_api.cu",
           "dact_ckpt.cu", "residual_norm_fwd.cu", "residual_norm_bwd.cu", "dense_residual_grad.cu", "dense_few.cu", "grad_norm.cu",
           "residual_api.cu"]
TENSOR_SOURCE = "tensor_list.cpp"
TENSOR_LIB_PATH = os.path.join(HERE, f"libte_gb300_tensors-{sys.implementation.cache_tag}-torch{torch.__version__}.so")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def _inputs():
    files = [os.path.join(CSRC, s) for s in SOURCES + [TENSOR_SOURCE]]
    files += [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith((".cuh", ".h"))]
    files += [os.path.join(INCLUDE, f) for f in os.listdir(INCLUDE)]
    files.append(os.path.abspath(__file__))
    return files


def up_to_date() -> bool:
    if not os.path.exists(LIB_PATH) or not os.path.exists(TENSOR_LIB_PATH):
        return False
    t = min(os.path.getmtime(LIB_PATH), os.path.getmtime(TENSOR_LIB_PATH))
    return all(os.path.getmtime(f) <= t for f in _inputs())


def build(verbose: bool = False, force: bool = False, ptxas_verbose: bool = False) -> str:
    if not force and up_to_date():
        return LIB_PATH
    os.makedirs(BUILD_DIR, exist_ok=True)
    cc = nvcc()
    common = ARCH + ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-I", INCLUDE,
                     "-I", CSRC]
    if ptxas_verbose:
        common += ["-Xptxas", "-v"]

    home = os.path.dirname(torch.__file__)
    tensors = ["-O2", "-std=c++17", "-Xcompiler", "-fPIC", "-I", INCLUDE, "-I", os.path.join(home, "include"), "-I",
               os.path.join(home, "include", "torch", "csrc", "api", "include"), "-I",
               sysconfig.get_paths()["include"], f"-D_GLIBCXX_USE_CXX11_ABI={int(torch.compiled_with_cxx11_abi())}"]

    def run(what, cmd):
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0 or verbose or ptxas_verbose:
            sys.stderr.write(" ".join(cmd) + "\n" + r.stdout + r.stderr)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {what}")

    def compile_one(src):
        obj = os.path.join(BUILD_DIR, os.path.splitext(src)[0] + ".o")
        run(src, [cc, *(tensors if src == TENSOR_SOURCE else common), "-c", os.path.join(CSRC, src), "-o", obj])
        return obj

    def link(path, args):
        tmp = path + ".tmp"
        run(os.path.basename(path), [cc, "-shared", "-o", tmp, *args])
        os.replace(tmp, path)

    with ThreadPoolExecutor(max_workers=len(SOURCES) + 1) as ex:
        tensor_obj = ex.submit(compile_one, TENSOR_SOURCE)
        objs = list(ex.map(compile_one, SOURCES))
        tensor_obj = tensor_obj.result()
    libs = os.path.join(home, "lib")
    link(TENSOR_LIB_PATH, [tensor_obj, "-cudart", "none", "-L", libs, "-lc10", "-ltorch_cpu", "-ltorch_python",
                           "-Xlinker", "-rpath," + libs])
    link(LIB_PATH, [*ARCH, *objs])
    return LIB_PATH


if __name__ == "__main__":
    build(verbose="-v" in sys.argv, force="-f" in sys.argv, ptxas_verbose="--ptxas" in sys.argv)
    print(LIB_PATH)
