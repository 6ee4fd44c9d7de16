"""Build the CUDA library in-tree: global_attention_b200/libzgcm_attn.so (sm_100a only).

    python -m global_attention_b200.build [--verbose]

Each csrc/*.cu is compiled by nvcc for sm_100a (objects under _build/), then linked into
one shared library with the CUDA runtime linked statically: nvcc is all it takes.  Where torch is installed,
csrc/torch_calls.cpp, the binding's quick calls, becomes the extension module global_attention_b200/_calls.so against the
library and torch (g++, torch's and Python's headers); it is built again when torch or Python is another one.  Where it
cannot be built the reason is printed, the library stands, and the calls that need the module raise.
"""
from __future__ import annotations

import glob
import os
import subprocess
import sys
import sysconfig
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
OBJ = os.path.join(ROOT, "_build")
LIB = os.path.join(HERE, "libzgcm_attn.so")
CALLS = os.path.join(HERE, "_calls.so")
CALLS_FOR = os.path.join(OBJ, "_calls.for")   # the torch and the Python it was built for
CXX = os.environ.get("CXX", "g++")
NVCC = os.environ.get("NVCC", "/usr/local/cuda/bin/nvcc")

FLAGS = ["-gencode", "arch=compute_100a,code=sm_100a", "-O3", "-lineinfo", "-std=c++17",
         "-Xcompiler", "-fPIC", "-I", os.path.join(ROOT, "include")]


def _needs(target: str, deps) -> bool:
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(d) > t for d in deps)


def build(verbose: bool = False, force: bool = False) -> str:
    os.makedirs(OBJ, exist_ok=True)
    srcs = sorted(glob.glob(os.path.join(CSRC, "*.cu")))
    headers = glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(ROOT, "include", "*.h"))

    def compile_one(src):
        obj = os.path.join(OBJ, os.path.basename(src)[:-3] + ".o")
        if force or _needs(obj, [src] + headers + [__file__]):
            cmd = [NVCC, *FLAGS, "-c", src, "-o", obj]
            if verbose:
                cmd.insert(1, "-Xptxas=-v")
            r = subprocess.run(cmd, capture_output=True, text=True)
            if r.returncode != 0:
                raise RuntimeError(f"nvcc failed on {src}:\n{r.stdout}\n{r.stderr}")
            if verbose:
                sys.stderr.write(r.stderr)
        return obj

    with ThreadPoolExecutor(max_workers=max(1, min(8, os.cpu_count() or 1))) as ex:
        objs = list(ex.map(compile_one, srcs))
    if force or _needs(LIB, objs):
        cmd = [NVCC, "-shared", "-gencode", "arch=compute_100a,code=sm_100a", "-cudart", "static",
               "-o", LIB + ".tmp", *objs, "-lcuda"]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
        os.replace(LIB + ".tmp", LIB)
    try:
        build_calls(force)
    except (ImportError, OSError, RuntimeError) as e:
        sys.stderr.write(f"{CALLS} is not built, the calls that need it will raise: {e}\n")
    return LIB


def build_calls(force: bool = False) -> str:
    """The extension module of csrc/torch_calls.cpp (host code; the library beside it is found by $ORIGIN)."""
    import torch
    src = os.path.join(CSRC, "torch_calls.cpp")
    wanted = f"torch {torch.__version__}, Python {sysconfig.get_config_var('SOABI')}"
    there = ""
    if os.path.exists(CALLS_FOR):
        with open(CALLS_FOR) as f:
            there = f.read()
    if force or there != wanted or _needs(CALLS, [src, __file__, *glob.glob(os.path.join(ROOT, "include", "*.h"))]):
        for old in (CALLS_FOR, CALLS):   # not to be taken for the new one if that fails
            if os.path.exists(old):
                os.remove(old)
        base = os.path.dirname(torch.__file__)
        inc = [os.path.join(ROOT, "include"), os.path.join(base, "include"),
               os.path.join(base, "include", "torch", "csrc", "api", "include"),
               os.path.join(os.path.dirname(os.path.dirname(NVCC)), "include"), sysconfig.get_paths()["include"]]
        cmd = [CXX, "-O2", "-std=c++17", "-fPIC", "-shared", "-w", *("-I" + d for d in inc),
               f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", src, "-o", CALLS + ".tmp",
               "-L" + os.path.join(base, "lib"), "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_python", "-ltorch",
               "-L" + HERE, "-l:" + os.path.basename(LIB), "-Wl,-rpath,$ORIGIN"]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"{CXX} failed on {src}:\n{r.stdout}\n{r.stderr}")
        os.replace(CALLS + ".tmp", CALLS)
        with open(CALLS_FOR, "w") as f:
            f.write(wanted)
    return CALLS


if __name__ == "__main__":
    print(build(verbose="--verbose" in sys.argv, force="--force" in sys.argv))
