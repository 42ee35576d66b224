"""Build libdecattn.so in-tree with nvcc for sm_103a, and the binding's calls.

Each .cu translation unit under csrc/ is compiled in parallel to an object
file, then linked into gqa_mqa_mla_gb300/lib/libdecattn.so (static cudart,
so the library needs only the driver at run time).  csrc/torch_calls.cpp, the
native half of the Python binding, is compiled beside them against PyTorch's
headers into lib/_calls.so.  Rebuilds are skipped when no source or header is
newer than both.
"""
from __future__ import annotations

import concurrent.futures as cf
import glob
import os
import shutil
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(PKG, "_build")
LIB_DIR = os.path.join(PKG, "lib")
LIB = os.path.join(LIB_DIR, "libdecattn.so")
CALLS = os.path.join(LIB_DIR, "_calls.so")
CALLS_SRC = os.path.join(CSRC, "torch_calls.cpp")
CALLS_FOR = CALLS + ".for"  # the PyTorch that _calls.so was compiled against

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-Xcompiler", "-O2",
              "--expt-relaxed-constexpr", f"-I{INCLUDE}", f"-I{CSRC}"]


def _nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: libdecattn needs the CUDA toolkit to build")


def sources() -> list[str]:
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _inputs() -> list[str]:
    return sources() + [CALLS_SRC] + glob.glob(os.path.join(CSRC, "*.h")) + glob.glob(
        os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(INCLUDE, "*.h")) + [__file__]


def calls_match() -> bool:
    """Was _calls.so compiled against the PyTorch that is installed?"""
    import torch

    try:
        with open(CALLS_FOR) as f:
            return f.read() == torch.__version__
    except OSError:
        return False


def up_to_date() -> bool:
    if not os.path.exists(LIB) or not os.path.exists(CALLS) or not calls_match():
        return False
    t = min(os.path.getmtime(LIB), os.path.getmtime(CALLS))
    return all(os.path.getmtime(f) <= t for f in _inputs())


def _build_calls() -> None:
    import sysconfig

    import torch

    cuda = os.path.dirname(os.path.dirname(os.path.realpath(_nvcc())))
    torch_dir = os.path.dirname(torch.__file__)
    tmp = CALLS + f".tmp{os.getpid()}"
    cmd = [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-shared",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", f"-I{INCLUDE}",
           f"-I{os.path.join(torch_dir, 'include')}",
           f"-I{os.path.join(torch_dir, 'include', 'torch', 'csrc', 'api', 'include')}",
           f"-I{sysconfig.get_paths()['include']}",
           f"-I{os.path.join(cuda, 'include')}", CALLS_SRC, "-o", tmp, f"-L{os.path.join(torch_dir, 'lib')}",
           "-ltorch_python", "-ltorch_cpu", "-lc10_cuda", "-lc10", "-ldl"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed on {CALLS_SRC}:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, CALLS)
    with open(CALLS_FOR, "w") as f:
        f.write(torch.__version__)


def build(force: bool = False, verbose: bool = False) -> str:
    if not force and up_to_date():
        return LIB
    nvcc = _nvcc()
    os.makedirs(BUILD, exist_ok=True)
    os.makedirs(LIB_DIR, exist_ok=True)

    def compile_one(src: str) -> str:
        obj = os.path.join(BUILD, os.path.basename(src)[:-3] + ".o")
        cmd = [nvcc, *ARCH, *NVCC_FLAGS, "-c", src, "-o", obj]
        if verbose:
            cmd.insert(1, "-Xptxas=-v")
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {src}:\n{r.stdout}\n{r.stderr}")
        if verbose and (r.stdout or r.stderr):
            sys.stderr.write(r.stdout + r.stderr)
        return obj

    with cf.ThreadPoolExecutor(max_workers=min(9, (os.cpu_count() or 4) + 1)) as ex:
        calls = ex.submit(_build_calls)
        objs = list(ex.map(compile_one, sources()))
        calls.result()
    tmp = LIB + f".tmp{os.getpid()}"
    # Static cudart; the driver's tensor-map encoder is resolved at run time
    # through cudaGetDriverEntryPointByVersion, so libcuda is not linked.
    cmd = [nvcc, *ARCH, "-shared", "-o", tmp, *objs, "-cudart", "static"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
