"""Builds the in-tree CUDA library ``libiq.so`` for sm_103a with nvcc.

Usage: ``python -m fp4_fp8_quant_gb300.build [--force] [--verbose]``.  The
translation units compile in parallel; the shared library links the CUDA
runtime statically, so it needs only the driver at run time.  Beside it stands
_iq_torch, the part of the Python binding that is written in C++ (g++ with
PyTorch's headers).  It is compiled for one PyTorch and one Python and fits no
other, so its file name says which: after a change of either it is built again.
"""

from __future__ import annotations

import os
import shutil
import subprocess
import sys
import sysconfig
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD_DIR = os.path.join(PKG, "_build")
LIB_PATH = os.path.join(PKG, "libiq.so")
BINDING_SOURCE = os.path.join(CSRC, "iq_torch.cpp")

SOURCES = ["iq_api.cu", "iq_quant.cu", "iq_gemm.cu", "iq_small_m.cu", "iq_indexer.cu", "iq_kv_cache.cu", "iq_kv_attention.cu",
           "iq_kv_attention_rows.cu", "iq_rows.cu", "iq_moe.cu",
           "iq_grouped.cu", "iq_adapters.cu"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-Xcompiler", "-O2",
              "--expt-relaxed-constexpr", f"-I{INCLUDE}", f"-I{CSRC}"]


def binding_path(torch_version: str | None = None) -> str:
    """The C++ module of the Python binding, for this Python and a PyTorch (the
    installed one)."""
    if torch_version is None:
        import torch
        torch_version = torch.__version__
    return os.path.join(PKG, f"_iq_torch.torch-{torch_version}{sysconfig.get_config_var('EXT_SUFFIX')}")


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libiq.so")


def _inputs():
    files = [os.path.join(CSRC, s) for s in SOURCES]
    files += [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith((".cuh", ".h"))]
    files += [os.path.join(INCLUDE, "iq.h"), BINDING_SOURCE]
    files.append(os.path.abspath(__file__))
    return files


def up_to_date() -> bool:
    built = (LIB_PATH, binding_path())
    if not all(map(os.path.exists, built)):
        return False
    t = min(map(os.path.getmtime, built))
    return all(os.path.getmtime(f) <= t for f in _inputs())


def _run(cmd, what: str) -> None:
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"{what} failed:\n{r.stdout}\n{r.stderr}")


def _build_binding() -> None:
    import torch
    root = os.path.dirname(torch.__file__)
    cuda = os.path.dirname(os.path.dirname(nvcc()))
    includes = [os.path.join(root, "include"), os.path.join(root, "include", "torch", "csrc", "api", "include"),
                os.path.join(cuda, "include"), sysconfig.get_paths()["include"]]
    path = binding_path()
    tmp = path + ".tmp"
    _run([os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-shared", *[f"-I{i}" for i in includes],
          f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", BINDING_SOURCE, "-o", tmp,
          f"-L{os.path.join(root, 'lib')}", "-ltorch_python", "-ltorch", "-ltorch_cpu", "-ltorch_cuda", "-lc10", "-lc10_cuda"], "g++ on iq_torch.cpp")
    os.replace(tmp, path)


def build(force: bool = False, verbose: bool = False) -> str:
    if not force and up_to_date():
        return LIB_PATH
    os.makedirs(BUILD_DIR, exist_ok=True)
    cc = nvcc()

    def compile_one(src):
        obj = os.path.join(BUILD_DIR, src.replace(".cu", ".o"))
        cmd = [cc, *ARCH, *NVCC_FLAGS, "-c", os.path.join(CSRC, src), "-o", obj]
        if verbose:
            cmd.insert(1, "-Xptxas=-v")
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {src}:\n{r.stdout}\n{r.stderr}")
        if verbose and (r.stdout or r.stderr):
            print(r.stdout + r.stderr, file=sys.stderr)
        return obj

    with ThreadPoolExecutor(max_workers=len(SOURCES) + 1) as ex:
        binding = ex.submit(_build_binding)
        objs = list(ex.map(compile_one, SOURCES))
        binding.result()
    tmp = LIB_PATH + ".tmp"
    _run([cc, *ARCH, "-shared", "-o", tmp, *objs], "link of libiq.so")
    os.replace(tmp, LIB_PATH)
    return LIB_PATH


if __name__ == "__main__":
    path = build(force="--force" in sys.argv, verbose="--verbose" in sys.argv)
    print(path)
