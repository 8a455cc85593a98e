"""Build libgret.so (the C-ABI CUDA library) in-tree for sm_100a with nvcc, and with g++ _paged.so,
the Python side of the paged cache's calls, against it and the installed torch.

    python gated_retention_linear_b200/build.py [--force] [--verbose]

(run by path: importing the package first would load the library being rebuilt)

Each csrc/*.cu compiles to an object under _build/ (in parallel, rebuilt when it or any header
is newer), then the objects link into gated_retention_linear_b200/libgret.so with the CUDA
runtime linked statically.  The driver API entry point for TMA descriptors is fetched at run
time through the runtime, so the library does not link libcuda.
"""
import concurrent.futures as cf
import glob
import importlib.metadata
import importlib.util
import os
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libgret.so")
BINDING = os.path.join(PKG, "_paged.so")
INCLUDE = os.path.join(ROOT, "include")

NVCC = os.environ.get("NVCC", "/usr/local/cuda/bin/nvcc")
ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "-Xcompiler", "-Wall",
         "--expt-relaxed-constexpr", "-I", INCLUDE, "-I", CSRC]


def _headers():
    return glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(INCLUDE, "*.h"))


def _stale(out, deps):
    if not os.path.exists(out):
        return True
    t = os.path.getmtime(out)
    return any(os.path.getmtime(d) > t for d in deps)


def _compile(src, verbose):
    obj = os.path.join(BUILD, os.path.basename(src)[:-3] + ".o")
    cmd = [NVCC] + ARCH + FLAGS + (["-Xptxas", "-v"] if verbose else []) + ["-c", src, "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("nvcc failed for %s:\n%s\n%s" % (src, r.stdout, r.stderr))
    return obj, r.stderr


def _build_binding(force):
    src = os.path.join(CSRC, "paged_binding.cpp")
    # whose C++ interfaces the binding is compiled against: neither is stable from one to the next
    tag = "torch %s, %s" % (importlib.metadata.version("torch"), sysconfig.get_config_var("SOABI"))
    tag_file = os.path.join(BUILD, "paged_binding.tag")
    if not force and not _stale(BINDING, [src, os.path.join(INCLUDE, "gret.h")]) \
            and os.path.exists(tag_file):
        with open(tag_file) as f:
            if f.read() == tag:
                return
    torch = os.path.dirname(importlib.util.find_spec("torch").origin)
    inc = [os.path.join(torch, "include"), sysconfig.get_paths()["include"], INCLUDE,
           os.path.join(os.path.dirname(os.path.dirname(NVCC)), "include")]
    tmp = BINDING + ".tmp.%d" % os.getpid()
    subprocess.run([os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-Wall", "-fPIC", "-shared",
                    "-fvisibility=hidden"] + ["-I" + i for i in inc]
                   + [src, "-o", tmp, "-L" + os.path.join(torch, "lib"), "-ltorch_python",
                      "-ltorch_cpu", "-lc10", "-lc10_cuda", "-L" + PKG, "-l:" + os.path.basename(LIB),
                      "-Wl,-rpath,$ORIGIN"], check=True)
    os.replace(tmp, BINDING)
    with open(tag_file, "w") as f:
        f.write(tag)


def build(force: bool = False, verbose: bool = False) -> str:
    os.makedirs(BUILD, exist_ok=True)
    srcs = sorted(glob.glob(os.path.join(CSRC, "*.cu")))
    hdrs = _headers()
    todo = [s for s in srcs
            if force or _stale(os.path.join(BUILD, os.path.basename(s)[:-3] + ".o"), [s] + hdrs)]
    with cf.ThreadPoolExecutor(max_workers=min(8, max(1, len(todo)))) as ex:
        for obj, log in ex.map(lambda s: _compile(s, verbose), todo):
            if verbose and log:
                sys.stderr.write(log)
    objs = [os.path.join(BUILD, os.path.basename(s)[:-3] + ".o") for s in srcs]
    if force or todo or _stale(LIB, objs):
        tmp = LIB + ".tmp.%d" % os.getpid()
        cmd = [NVCC] + ARCH + ["-shared", "-cudart", "static", "-o", tmp] + objs
        subprocess.run(cmd, check=True)
        os.replace(tmp, LIB)
    _build_binding(force)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="--verbose" in sys.argv))
