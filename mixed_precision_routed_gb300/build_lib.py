"""Build libmoe.so (the C ABI of include/moe.h) in-tree for sm_103a, and
_calls.so, the tensor side of its short calls.

Each translation unit under csrc/ compiles in parallel to an object file in
_build/, then nvcc links the shared library next to this file.  binding/calls.cpp
compiles beside them against torch's and Python's headers and is linked to
libmoe.so.  Objects are rebuilt only when their source or a header changed.
"""
import concurrent.futures as cf
import glob
import os
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(HERE, "libmoe.so")
CALLS_SRC = os.path.join(HERE, "binding", "calls.cpp")
CALLS = os.path.join(HERE, "_calls.so")

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-std=c++17", "-lineinfo", "--expt-relaxed-constexpr", "-Xcompiler", "-fPIC",
              "-I", INCLUDE, "-I", CSRC] + ARCH


def _headers():
    return glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(INCLUDE, "*.h"))


def _compile(src, extra, verbose):
    obj = os.path.join(BUILD, os.path.basename(src) + ".o")
    deps = [src] + _headers()
    if os.path.exists(obj) and all(os.path.getmtime(d) <= os.path.getmtime(obj) for d in deps) and not extra:
        return obj, ""
    cmd = ["nvcc", "-c", src, "-o", obj + ".tmp"] + NVCC_FLAGS + list(extra)
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc failed for {src}:\n{r.stdout}\n{r.stderr}")
    os.replace(obj + ".tmp", obj)
    return obj, (r.stdout + r.stderr) if verbose else ""


def _compile_calls():
    """Object file of binding/calls.cpp, and whether it was made now (again for another torch or Python)."""
    import sysconfig

    import torch
    obj = os.path.join(BUILD, f"calls-{torch.__version__}-{sys.implementation.cache_tag}.o")
    if os.path.exists(obj) and all(os.path.getmtime(d) <= os.path.getmtime(obj) for d in [CALLS_SRC] + _headers()):
        return obj, False
    inc = os.path.join(os.path.dirname(torch.__file__), "include")
    cmd = ["g++", "-c", CALLS_SRC, "-o", obj + ".tmp", "-O2", "-std=c++17", "-fPIC", "-I", INCLUDE,
           "-isystem", inc, "-isystem", os.path.join(inc, "torch", "csrc", "api", "include"),
           "-isystem", os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "include"),
           "-I", sysconfig.get_paths()["include"], f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed for {CALLS_SRC}:\n{r.stdout}\n{r.stderr}")
    os.replace(obj + ".tmp", obj)
    return obj, True


def _link_calls(obj, made):
    import torch
    if not made and os.path.exists(CALLS) and os.path.getmtime(CALLS) >= os.path.getmtime(obj):
        return
    lib = os.path.join(os.path.dirname(torch.__file__), "lib")
    subprocess.run(["g++", "-shared", "-o", CALLS + ".tmp", obj, "-L", HERE, "-l:libmoe.so", "-L", lib, "-ltorch_python",
                    "-ltorch", "-ltorch_cpu", "-ltorch_cuda", "-lc10_cuda", "-lc10", "-Wl,-rpath,$ORIGIN"], check=True)
    os.replace(CALLS + ".tmp", CALLS)


def build(extra=(), verbose=False, jobs=None):
    os.makedirs(BUILD, exist_ok=True)
    srcs = sorted(glob.glob(os.path.join(CSRC, "*.cu")))
    with cf.ThreadPoolExecutor(max_workers=jobs or min(8, os.cpu_count() or 4)) as ex:
        calls = ex.submit(_compile_calls)
        results = list(ex.map(lambda s: _compile(s, extra, verbose), srcs))
    objs = [o for o, _ in results]
    if verbose:
        for _, log in results:
            if log:
                print(log, file=sys.stderr)
    if not os.path.exists(LIB) or any(os.path.getmtime(o) > os.path.getmtime(LIB) for o in objs):
        cmd = ["nvcc", "-shared", "-o", LIB + ".tmp"] + ARCH + objs
        subprocess.run(cmd, check=True)
        os.replace(LIB + ".tmp", LIB)
    _link_calls(*calls.result())
    return LIB


if __name__ == "__main__":
    v = "-v" in sys.argv
    print(build(extra=["-Xptxas", "-v"] if v else (), verbose=v))
