"""Build ``libne_attn.so`` in-tree with nvcc for sm_103a (GB300), and the module
``ne_step`` that makes a generation step's calls from Python.

The translation units are compiled in parallel, then linked into
``causal_self_attention_gb300/_build/libne_attn.so``.  No CMake, no torch
extension machinery: the library is plain C ABI (include/ne_attn.h).  The module
alone knows torch's tensors; it is built for the torch that is installed.
"""
from __future__ import annotations

import os
import shutil
import subprocess
import sys
import sysconfig
import warnings
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
BUILD_DIR = os.path.join(HERE, "_build")
LIB_PATH = os.path.join(BUILD_DIR, "libne_attn.so")
SOURCES = ["ne_attn_api.cu", "ne_attn_fwd.cu", "ne_attn_gqa_fwd.cu", "ne_attn_bwd.cu", "ne_attn_noalloc.cu",
           "ne_attn_decode.cu", "ne_attn_paged.cu", "ne_kv_cache.cu", "ne_kv_pages.cu", "ne_qk_norm.cu", "ne_debug.cu", "ne_proj.cu", "ne_sched.cu"]
STEP_SOURCE = "ne_step.cpp"
GENCODE = "-gencode=arch=compute_103a,code=sm_103a"


def nvcc_path() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def _deps_mtime() -> float:
    paths = [os.path.join(CSRC, f) for f in os.listdir(CSRC)]
    paths += [os.path.join(ROOT, "include", f) for f in os.listdir(os.path.join(ROOT, "include"))]
    paths.append(os.path.abspath(__file__))
    return max(os.path.getmtime(p) for p in paths)


def compile_flags(extra=()) -> list:
    return [GENCODE, "-O3", "-lineinfo", "-std=c++17", "--expt-relaxed-constexpr",
            "-Xcompiler", "-fPIC", "-I" + os.path.join(ROOT, "include"), *extra]


def step_path() -> str:
    """The path of the module ``ne_step`` for this torch and this interpreter's ABI."""
    import torch
    suffix = sysconfig.get_config_var("EXT_SUFFIX")
    return os.path.join(BUILD_DIR, f"ne_step-{torch.__version__}{suffix}")


def _cuda_include() -> str:
    """The folder of CUDA's headers (of the runtime, which torch's name)."""
    nvcc = os.environ.get("NVCC") or shutil.which("nvcc")
    homes = [os.environ.get("CUDA_HOME"), os.environ.get("CUDA_PATH"),
             nvcc and os.path.dirname(os.path.dirname(os.path.realpath(nvcc))), "/usr/local/cuda"]
    for home in filter(None, homes):
        if os.path.exists(os.path.join(home, "include", "cuda_runtime_api.h")):
            return os.path.join(home, "include")
    raise RuntimeError("cuda_runtime_api.h not found (CUDA_HOME names where CUDA is)")


def _build_step(path: str) -> None:
    import torch
    home = os.path.dirname(torch.__file__)
    include = (os.path.join(home, "include"),
               os.path.join(home, "include", "torch", "csrc", "api", "include"),
               sysconfig.get_paths()["include"], _cuda_include(), os.path.join(ROOT, "include"))
    tmp = path + f".tmp{os.getpid()}"
    cmd = [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-shared", "-fPIC",
           *("-I" + d for d in include), os.path.join(CSRC, STEP_SOURCE), "-o", tmp,
           "-L" + os.path.join(home, "lib"), "-ltorch_python", "-ltorch_cpu", "-lc10", "-lc10_cuda"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"{cmd[0]} failed for {STEP_SOURCE}:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, path)


def build(force: bool = False, verbose: bool = False, ptxas_info: bool = False) -> str:
    """Compile (if stale) and return the library path.  Where the module cannot be built, a
    warning says so: the binding makes its calls itself then."""
    os.makedirs(BUILD_DIR, exist_ok=True)
    step, deps = step_path(), _deps_mtime()
    fresh = [not force and os.path.exists(p) and os.path.getmtime(p) >= deps for p in (LIB_PATH, step)]
    with ThreadPoolExecutor(max_workers=1) as ex:
        module = None if fresh[1] else ex.submit(_build_step, step)
        if not fresh[0]:
            _build_library(verbose, ptxas_info)
        if module is not None:
            try:
                module.result()
            except (RuntimeError, OSError) as e:
                if os.path.exists(step):  # (one of older sources)
                    os.remove(step)
                warnings.warn(f"the module ne_step is not built, calls are marshalled in Python: {e}",
                              RuntimeWarning, stacklevel=2)
    return LIB_PATH


def _build_library(verbose: bool, ptxas_info: bool) -> None:
    nvcc = nvcc_path()
    extra = ["-Xptxas", "-v"] if ptxas_info else []

    def compile_one(src):
        obj = os.path.join(BUILD_DIR, src.replace(".cu", ".o"))
        cmd = [nvcc, *compile_flags(extra), "-c", os.path.join(CSRC, src), "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed for {src}:\n{r.stdout}\n{r.stderr}")
        if verbose or ptxas_info:
            sys.stderr.write(r.stdout + r.stderr)
        return obj

    with ThreadPoolExecutor(max_workers=len(SOURCES)) as ex:
        objs = list(ex.map(compile_one, SOURCES))
    tmp = LIB_PATH + f".tmp{os.getpid()}"
    cmd = [nvcc, GENCODE, "-shared", "-o", tmp, *objs]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB_PATH)


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose=True, ptxas_info="--ptxas" in sys.argv)
    print(LIB_PATH)
