"""Builds ``libpkv.so`` (the C-ABI library) in-tree with nvcc for sm_103a.

Translation units are compiled in parallel; the CUDA runtime is linked
statically so the library loads on machines without a GPU driver (host-only
entry points such as the page pool work there).  ``pkv_torch`` is a Python
module on top of it that checks tensors in C++ (g++, with torch's headers).
The library does not need it: where it cannot be built, the library is, and the
calls that go through the module say why.
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
    return [os.path.join(CSRC, s) for s in CUDA_SOURCES + CXX_SOURCES] + \
        [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith((".h", ".cuh"))] + \
        [os.path.join(INCLUDE, "pkv.h")]


def _newer(path: str, sources) -> bool:
    return os.path.exists(path) and all(os.path.getmtime(s) <= os.path.getmtime(path) for s in sources)


def up_to_date() -> bool:
    return _newer(LIB_PATH, _sources())


def module_path() -> str:
    """Where the Python module lies, under a name of its own for every torch and
    Python: one that was built for others is not loaded."""
    import torch

    return os.path.join(HERE, f"pkv_torch-{torch.__version__}{sysconfig.get_config_var('EXT_SUFFIX')}")


def module_up_to_date() -> bool:
    return _newer(module_path(), [os.path.join(CSRC, TORCH_SOURCE), os.path.join(INCLUDE, "pkv.h")])


def _run(cmd):
    return cmd, subprocess.run(cmd, capture_output=True, text=True)


def _good(step: str, result, verbose: bool = False) -> None:
    cmd, r = result
    if r.returncode != 0:
        raise RuntimeError(f"{step} failed: {' '.join(cmd)}\n{r.stdout}\n{r.stderr}")
    if verbose and (r.stdout or r.stderr):
        sys.stderr.write(r.stdout + r.stderr)


def _module_job():
    """Compile command of the Python module and how its object is linked."""
    import torch

    root = os.path.dirname(torch.__file__)
    obj = os.path.join(BUILD_DIR, "pkv_torch.o")
    cxx = shutil.which("g++") or "g++"
    cuda = os.path.join(os.path.dirname(os.path.dirname(_nvcc())), "include")
    compile_ = [cxx, "-O2", "-std=c++17", "-fPIC", "-fvisibility=hidden", "-Wall",
                f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", "-I", INCLUDE,
                "-isystem", os.path.join(root, "include"),
                "-isystem", os.path.join(root, "include", "torch", "csrc", "api", "include"),
                "-isystem", sysconfig.get_paths()["include"], "-isystem", cuda,
                "-c", os.path.join(CSRC, TORCH_SOURCE), "-o", obj]
    libs = os.path.join(root, "lib")
    link = [cxx, "-shared", "-o", None, obj, LIB_PATH, "-Wl,-rpath,$ORIGIN", f"-L{libs}", f"-Wl,-rpath,{libs}",
            "-ltorch_python", "-ltorch_cpu", "-lc10", "-lc10_cuda"]
    return compile_, link


def _link_module(link, verbose: bool) -> None:
    path = module_path()
    tmp = path + f".tmp{os.getpid()}"
    link[link.index(None)] = tmp
    _good("link", _run(link), verbose)
    os.replace(tmp, path)


def build_module(force: bool = False, verbose: bool = False) -> str:
    """Compile and link the Python module alone (the library is there); returns its
    path, or raises with what the compiler says."""
    if force or not module_up_to_date():
        os.makedirs(BUILD_DIR, exist_ok=True)
        compile_, link = _module_job()
        _good("compile", _run(compile_), verbose)
        _link_module(link, verbose)
    return module_path()


def build(force: bool = False, verbose: bool = False) -> str:
    """Compile and link the library, and the Python module if that can be built;
    returns the library path."""
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

    objs = [j[-1] for j in jobs]
    failure = None  # of the module
    try:
        module_compile, module_link = _module_job()
        jobs.append(module_compile)
    except Exception as e:  # (no torch, or one of another kind)
        failure = e

    with ThreadPoolExecutor(max_workers=len(jobs)) as ex:
        results = list(ex.map(_run, jobs))
    for result in results[:len(objs)]:
        _good("compile", result, verbose)
    tmp = LIB_PATH + f".tmp{os.getpid()}"
    _good("link", _run([nvcc, *ARCH, "-shared", "-cudart", "static", "-Xlinker", "-soname=libpkv.so", "-o", tmp, *objs]))
    os.replace(tmp, LIB_PATH)
    if failure is None:
        try:
            _good("compile", results[-1], verbose)
            _link_module(module_link, verbose)
        except Exception as e:
            failure = e
    if failure is not None:
        sys.stderr.write(f"pkv_torch was not built: {failure}\n")
    return LIB_PATH


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
