"""Build the C-ABI library ``libsconvkv.so`` (sm_100a) in-tree with nvcc, and
``_tree.so``, the Python module that marshals tensors for some of its calls, with g++.

The host code (``csrc/tree_ops.cu``, which includes ``csrc/sconv_kv.cu``) and
the kernel-instance translation units (``csrc/inst_*.cu``) are compiled to
objects in parallel, then linked into one shared library.
"""
import concurrent.futures
import os
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
HEADER = os.path.join(INCLUDE, "sconv_kv.h")
LIB = os.path.join(PKG, "libsconvkv.so")
TREE = os.path.join(PKG, "_tree.so")
TREE_SOURCE = os.path.join(CSRC, "tree_bind.cpp")
# tree_ops.cu includes sconv_kv.cu
SOURCES = [os.path.join(CSRC, "tree_ops.cu")] + sorted(
    os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.startswith("inst_") and f.endswith(".cu"))
DEPS = [os.path.join(CSRC, f) for f in os.listdir(CSRC)] + [
    os.path.join(INCLUDE, f) for f in os.listdir(INCLUDE)]

ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
COMPILE_FLAGS = ARCH + ["-O3", "-lineinfo", "-std=c++17", "-Xptxas", "-v",
                        "-Xcompiler", "-fPIC", "-Xcompiler", "-fvisibility=hidden"]


def nvcc():
    cand = os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "bin", "nvcc")
    return cand if os.path.exists(cand) else "nvcc"


def _older(out, deps):
    """Whether `out` is missing, or older than one of `deps`."""
    if not os.path.exists(out):
        return True
    t = os.path.getmtime(out)
    return any(os.path.getmtime(d) > t for d in deps if os.path.exists(d))


def needs_build(out=LIB):
    """Whether build(out) has something to do: the library, and beside its usual place the
    marshalling module."""
    return _older(out, DEPS) or (out == LIB and _older(TREE, [TREE_SOURCE, HEADER]))


def _compile(src, obj, extra):
    cmd = [nvcc(), *COMPILE_FLAGS, *extra, "-I", INCLUDE, "-I", CSRC, "-c", "-o", obj, src]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError("nvcc failed:\n" + " ".join(cmd) + "\n" + res.stdout + res.stderr)
    return res.stdout + res.stderr


def build_tree(out=TREE):
    """Compile and link the marshalling module against the installed torch."""
    import sysconfig

    import torch
    root = os.path.dirname(torch.__file__)
    libs = os.path.join(root, "lib")
    cuda = os.path.join(os.path.dirname(os.path.dirname(nvcc())), "include")
    inc = [INCLUDE, os.path.join(root, "include"),
           os.path.join(root, "include", "torch", "csrc", "api", "include"),
           sysconfig.get_paths()["include"], cuda]
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           *(f"-I{i}" for i in inc), TREE_SOURCE, "-o", out, f"-L{libs}", f"-Wl,-rpath,{libs}",
           "-lc10", "-lc10_cuda", "-ltorch", "-ltorch_cpu", "-ltorch_python"]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError("g++ failed:\n" + " ".join(cmd) + "\n" + res.stdout + res.stderr)
    return out


def build(out=LIB, quiet=True, extra=()):
    """Compile every translation unit (in parallel) and link `out`; the library's
    usual place gets the marshalling module beside it."""
    objdir = os.path.join(ROOT, "_build", os.path.basename(out) + ".objs")
    os.makedirs(objdir, exist_ok=True)
    objs = [os.path.join(objdir, os.path.basename(s)[:-3] + ".o") for s in SOURCES]
    workers = max(1, min(len(SOURCES) + 1, os.cpu_count() or 1))
    with concurrent.futures.ThreadPoolExecutor(max_workers=workers) as ex:
        tree = ex.submit(build_tree) if out == LIB else None
        logs = list(ex.map(lambda so: _compile(so[0], so[1], extra), zip(SOURCES, objs)))
        if tree:
            tree.result()
    cmd = [nvcc(), *ARCH, "-shared", "-o", out, *objs]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError("nvcc link failed:\n" + " ".join(cmd) + "\n" + res.stdout + res.stderr)
    with open(out + ".ptxas.txt", "w") as f:
        f.write("".join(logs) + res.stdout + res.stderr)
    if not quiet:
        sys.stderr.write("".join(logs))
    return out


if __name__ == "__main__":
    print(build(quiet=False))
