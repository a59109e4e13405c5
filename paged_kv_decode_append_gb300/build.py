"""Builds ``libpkv.so`` (the C-ABI library) in-tree with nvcc for sm_103a.

Translation units are compiled in parallel; the CUDA runtime is linked
statically so the library loads on machines without a GPU driver (host-only
entry points such as the page pool work there).  ``pkv_torch.so`` is a Python
module on top of it that checks tensors in C++ (g++, with torch's headers).
"""
from __future__ import annotations

import os
import shutil
import subprocess
import sys
import sysconfig
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD_DIR = os.path.join(HERE, "_build")
LIB_PATH = os.path.join(HERE, "libpkv.so")
TORCH_LIB_PATH = os.path.join(HERE, "pkv_torch.so")

CUDA_SOURCES = ["pkv_decode.cu", "pkv_prefill.cu", "pkv_append.cu", "pkv_api.cu", "pkv_static.cu",
                "pkv_table.cu", "pkv_tree.cu", "pkv_tree_attn.cu", "pkv_rope.cu", "pkv_mass.cu", "pkv_evict.cu"]
CXX_SOURCES = ["pkv_pool.cc", "pkv_graph.cc"]
TORCH_SOURCE = "pkv_torch.cc"  # a Python module over the library, with torch's headers
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]


def _nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def _sources():
    return [os.path.join(CSRC, s) for s in CUDA_SOURCES + CXX_SOURCES + [TORCH_SOURCE]] + \
        [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith((".h", ".cuh"))] + \
        [os.path.join(INCLUDE, "pkv.h")]


def up_to_date() -> bool:
    if not os.path.exists(LIB_PATH) or not os.path.exists(TORCH_LIB_PATH):
        return False
    t = min(os.path.getmtime(LIB_PATH), os.path.getmtime(TORCH_LIB_PATH))
    return all(os.path.getmtime(s) <= t for s in _sources())


def _torch_job():
    """Compile command of the Python module, its object and how it is linked."""
    import torch

    root = os.path.dirname(torch.__file__)
    obj = os.path.join(BUILD_DIR, "pkv_torch.o")
    cxx = shutil.which("g++") or "g++"
    cuda = os.path.join(os.path.dirname(os.path.dirname(_nvcc())), "include")
    compile_ = [cxx, "-O2", "-std=c++17", "-fPIC", "-fvisibility=hidden", "-w",
                f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", "-I", INCLUDE,
                "-isystem", os.path.join(root, "include"),
                "-isystem", os.path.join(root, "include", "torch", "csrc", "api", "include"),
                "-isystem", sysconfig.get_paths()["include"], "-isystem", cuda,
                "-c", os.path.join(CSRC, TORCH_SOURCE), "-o", obj]
    libs = os.path.join(root, "lib")
    link = [cxx, "-shared", "-o", None, obj, LIB_PATH, "-Wl,-rpath,$ORIGIN", f"-L{libs}", f"-Wl,-rpath,{libs}",
            "-ltorch_python", "-ltorch_cpu", "-lc10", "-lc10_cuda"]
    return compile_, link


def build(force: bool = False, verbose: bool = False) -> str:
    """Compile and link; returns the library path."""
    if not force and up_to_date():
        return LIB_PATH
    nvcc = _nvcc()
    os.makedirs(BUILD_DIR, exist_ok=True)
    common = ["-O3", "-std=c++17", "-I", INCLUDE, "-I", CSRC, "-Xcompiler", "-fPIC,-fvisibility=hidden"]
    jobs = []
    for s in CUDA_SOURCES:
        obj = os.path.join(BUILD_DIR, s.replace(".cu", ".o"))
        jobs.append([nvcc, *ARCH, "-lineinfo", *common, "-Xptxas", "-v" if verbose else "-O3",
                     "-c", os.path.join(CSRC, s), "-o", obj])
    for s in CXX_SOURCES:
        obj = os.path.join(BUILD_DIR, s.replace(".cc", ".o"))
        jobs.append([nvcc, *common, "-x", "c++", "-c", os.path.join(CSRC, s), "-o", obj])

    torch_compile, torch_link = _torch_job()
    jobs.append(torch_compile)

    def run(cmd):
        r = subprocess.run(cmd, capture_output=True, text=True)
        return cmd, r

    with ThreadPoolExecutor(max_workers=len(jobs)) as ex:
        results = list(ex.map(run, jobs))
    for cmd, r in results:
        if r.returncode != 0:
            raise RuntimeError(f"compile failed: {' '.join(cmd)}\n{r.stdout}\n{r.stderr}")
        if verbose and (r.stdout or r.stderr):
            sys.stderr.write(r.stdout + r.stderr)
    objs = [j[-1] for j in jobs[:-1]]
    tmp = LIB_PATH + f".tmp{os.getpid()}"
    link = [nvcc, *ARCH, "-shared", "-cudart", "static", "-Xlinker", "-soname=libpkv.so", "-o", tmp, *objs]
    r = subprocess.run(link, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed: {' '.join(link)}\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB_PATH)
    tmp = TORCH_LIB_PATH + f".tmp{os.getpid()}"
    torch_link[torch_link.index(None)] = tmp
    r = subprocess.run(torch_link, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed: {' '.join(torch_link)}\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, TORCH_LIB_PATH)
    return LIB_PATH


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
