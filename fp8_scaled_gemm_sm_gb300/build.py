"""Build libscaledgemm.so (the sm_103a kernels + C ABI) in-tree with nvcc, and the
attention operators' torch binding beside it.

Every .cu under csrc/ is compiled in parallel for
``-gencode arch=compute_103a,code=sm_103a`` and linked into
``fp8_scaled_gemm_sm_gb300/libscaledgemm.so`` with the CUDA runtime linked
statically, so the library loads on a machine without a GPU (its entry points
then return SG_ERR_CUDA).  ``_attn.so`` (host code, the C++ compiler and torch's
headers) is compiled at the same time and links to it.  The library does not depend
on it: without torch only the library is built, and where ``_attn.so`` does not build
the library is there before the error is raised.
"""
import importlib.util
import os
import shutil
import subprocess
import sys
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(ROOT, "_build")
LIB = os.path.join(PKG, "libscaledgemm.so")
EXT = os.path.join(PKG, "_attn.so")
EXT_SRC = os.path.join(CSRC, "sg_attn_torch.cpp")

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ARCH + [
    "-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-Xcompiler", "-Wall",
    "-I" + INCLUDE, "-I" + CSRC,
]


def nvcc():
    p = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(p):
        raise RuntimeError("nvcc not found")
    return p


def sources():
    return sorted(os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith(".cu"))


def _deps():
    return sources() + [EXT_SRC] + [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith((".cuh", ".h"))] + [
        os.path.join(INCLUDE, f) for f in os.listdir(INCLUDE) if f.endswith(".h")
    ] + [os.path.abspath(__file__)]


def have_torch():
    return importlib.util.find_spec("torch") is not None


def up_to_date():
    made = [LIB, EXT] if have_torch() else [LIB]
    if not all(os.path.exists(f) for f in made):
        return False
    t = min(os.path.getmtime(f) for f in made)
    return all(os.path.getmtime(d) <= t for d in _deps())


def build(force=False, verbose=False, extra_flags=()):
    """Compile and link the library unless it is newer than all its sources."""
    if not force and up_to_date():
        return LIB
    os.makedirs(BUILD, exist_ok=True)
    cc = nvcc()

    def compile_one(src):
        obj = os.path.join(BUILD, os.path.basename(src)[:-3] + ".o")
        cmd = [cc] + NVCC_FLAGS + list(extra_flags) + ["-c", src, "-o", obj]
        if verbose:
            print(" ".join(cmd), file=sys.stderr)
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError("nvcc failed for %s:\n%s%s" % (src, r.stdout, r.stderr))
        if verbose and (r.stdout or r.stderr):
            print(r.stdout + r.stderr, file=sys.stderr)
        return obj

    srcs = sources()
    with ThreadPoolExecutor(max_workers=max(1, min(len(srcs) + 1, os.cpu_count() or 4))) as ex:
        ext = ex.submit(_compile_ext, verbose) if have_torch() else None
        objs = list(ex.map(compile_one, srcs))
    tmp = LIB + ".tmp.%d" % os.getpid()
    cmd = [cc] + ARCH + ["-shared", "-Xcompiler", "-fPIC", "--cudart", "static", "-o", tmp] + objs
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("link failed:\n%s%s" % (r.stdout, r.stderr))
    os.replace(tmp, LIB)
    if ext is not None:
        _link_ext(ext.result())
    return LIB


def _run(cmd, what):
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("%s failed:\n%s%s" % (what, r.stdout, r.stderr))


def _torch_dirs():
    import torch

    root = os.path.dirname(torch.__file__)
    return root, int(torch._C._GLIBCXX_USE_CXX11_ABI)


def _compile_ext(verbose):
    import sysconfig

    torch_root, abi = _torch_dirs()
    obj = os.path.join(BUILD, "sg_attn_torch.o")
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(nvcc())))
    cmd = [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-D_GLIBCXX_USE_CXX11_ABI=%d" % abi, "-c", EXT_SRC, "-o", obj,
           "-I" + INCLUDE, "-isystem", os.path.join(torch_root, "include"),
           "-isystem", os.path.join(torch_root, "include", "torch", "csrc", "api", "include"),
           "-isystem", sysconfig.get_paths()["include"], "-isystem", os.path.join(cuda, "include")]
    if verbose:
        print(" ".join(cmd), file=sys.stderr)
    _run(cmd, "compiling " + EXT_SRC)
    return obj


def _link_ext(obj):
    libs = os.path.join(_torch_dirs()[0], "lib")
    tmp = EXT + ".tmp.%d" % os.getpid()
    _run([os.environ.get("CXX", "g++"), "-shared", "-o", tmp, obj, "-L" + PKG, "-l:" + os.path.basename(LIB), "-Wl,-rpath,$ORIGIN", "-L" + libs, "-Wl,-rpath," + libs,
          "-ltorch_python", "-ltorch_cpu", "-ltorch", "-lc10_cuda", "-lc10"], "linking " + EXT)
    os.replace(tmp, EXT)


if __name__ == "__main__":
    flags = [a for a in sys.argv[1:] if a.startswith("-X") or a.startswith("--")]
    print(build(force=True, verbose=True, extra_flags=[f for f in flags if f != "--force"]))
