"""Build libcsa.so (the C-ABI library) in-tree with nvcc for sm_100a.

    python -m fp4_compressed_sparse_kv_b200.build [--verbose-ptxas]

Each .cu under csrc/ is compiled to an object under _build/ and linked with a static CUDA runtime,
so the shared object loads wherever the NVIDIA driver is present.  csrc/run_binding.cpp, argument marshalling of the
Python binding against PyTorch's headers, becomes _runs.so.
"""
import argparse
import concurrent.futures as cf
import glob
import importlib.metadata
import importlib.util
import os
import shutil
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
BUILD = os.path.join(os.path.dirname(HERE), "_build")
LIB = os.path.join(HERE, "libcsa.so")
RUNS = os.path.join(HERE, "_runs.so")
RUNS_STAMP = os.path.join(BUILD, "_runs.stamp")   # what _runs.so was built against
INCLUDE = os.path.join(os.path.dirname(HERE), "include")

ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
NVCC_FLAGS = ARCH + ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC,-O2", "-I", INCLUDE,
                     "--expt-relaxed-constexpr", "-Werror", "all-warnings"]


def nvcc():
    exe = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(exe):
        raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libcsa.so")
    return exe


def _compile(src, verbose_ptxas):
    obj = os.path.join(BUILD, os.path.basename(src)[:-3] + ".o")
    deps = [src] + glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(INCLUDE, "*.h"))
    if os.path.exists(obj) and os.path.getmtime(obj) >= max(os.path.getmtime(d) for d in deps) \
            and not verbose_ptxas:
        return obj, ""
    cmd = [nvcc(), *NVCC_FLAGS, "-c", src, "-o", obj]
    if verbose_ptxas:
        cmd += ["-Xptxas", "-v"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("nvcc failed for %s:\n%s%s" % (src, r.stdout, r.stderr))
    return obj, r.stderr


def _build_binding():
    src = os.path.join(CSRC, "run_binding.cpp")
    deps = [src, os.path.join(INCLUDE, "csa.h")]
    # PyTorch's C++ interface and Python's differ from version to version
    version = importlib.metadata.version("torch")
    stamp = "torch %s\npython %s\n" % (version, sys.version)
    if os.path.exists(RUNS) and os.path.getmtime(RUNS) >= max(os.path.getmtime(d) for d in deps) \
            and os.path.exists(RUNS_STAMP) and open(RUNS_STAMP).read() == stamp:
        return
    torch = os.path.dirname(importlib.util.find_spec("torch").origin)
    cuda = os.path.dirname(os.path.dirname(nvcc()))
    tmp = RUNS + ".tmp.%d" % os.getpid()
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-Wall", "-Werror", "-I", INCLUDE,
           '-DCSA_TORCH_VERSION="%s"' % version]
    for inc in (os.path.join(torch, "include"), sysconfig.get_paths()["include"], os.path.join(cuda, "include")):
        cmd += ["-isystem", inc]
    cmd += [src, "-o", tmp, "-L", os.path.join(torch, "lib"), "-ltorch_python", "-ltorch_cpu", "-lc10", "-lc10_cuda"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("g++ failed for %s:\n%s%s" % (src, r.stdout, r.stderr))
    os.replace(tmp, RUNS)
    with open(RUNS_STAMP, "w") as f:
        f.write(stamp)


def build(verbose_ptxas: bool = False, quiet: bool = True) -> str:
    os.makedirs(BUILD, exist_ok=True)
    srcs = sorted(glob.glob(os.path.join(CSRC, "*.cu")))
    with cf.ThreadPoolExecutor(max_workers=min(8, len(srcs))) as ex:
        results = list(ex.map(lambda s: _compile(s, verbose_ptxas), srcs))
    objs = [o for o, _ in results]
    if verbose_ptxas or not quiet:
        for _, log in results:
            if log:
                sys.stderr.write(log)
    newest = max(os.path.getmtime(o) for o in objs)
    if not os.path.exists(LIB) or os.path.getmtime(LIB) < newest:
        tmp = LIB + ".tmp.%d" % os.getpid()
        cmd = [nvcc(), *ARCH, "-shared", "-cudart", "static", "-o", tmp, *objs]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError("link failed:\n%s%s" % (r.stdout, r.stderr))
        os.replace(tmp, LIB)
    _build_binding()
    return LIB


if __name__ == "__main__":
    ap = argparse.ArgumentParser()
    ap.add_argument("--verbose-ptxas", action="store_true")
    args = ap.parse_args()
    print(build(verbose_ptxas=args.verbose_ptxas, quiet=False))
