"""Builds the CUDA library ``libw8lin.so`` in-tree for sm_103a.

Each translation unit under ``csrc/`` is compiled in parallel with nvcc,
then linked into one shared library next to this file.  Objects go to
``_build/``.  Rebuilds only what changed (source, header or flags newer than
the object).
"""

import concurrent.futures as cf
import os
import shutil
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
OUT_DIR = os.path.join(HERE, "_build")
LIB = os.path.join(HERE, "libw8lin.so")
SOURCES = ["api.cu", "attention.cu", "elementwise.cu", "gemm.cu", "noalloc.cu", "paged_attention.cu", "paged_few.cu", "policy.cu",
           "rmsnorm.cu", "rope.cu"]

MARSHAL = os.path.join(HERE, "_marshal.so")
MARSHAL_FOR = os.path.join(OUT_DIR, "marshal.txt")   # the PyTorch and Python that it was compiled with

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ARCH + ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC",
                     "-Xcompiler", "-fno-strict-aliasing", "--expt-relaxed-constexpr"]


def _nvcc():
    cand = [os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"]
    for c in cand:
        if c and os.path.exists(c):
            return c
    raise RuntimeError("nvcc not found")


def _headers():
    hs = [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith((".cuh", ".h"))]
    hs.append(os.path.join(ROOT, "include", "w8lin.h"))
    hs.append(os.path.abspath(__file__))
    return hs


def _stale(obj, deps):
    if not os.path.exists(obj):
        return True
    t = os.path.getmtime(obj)
    return any(os.path.getmtime(d) > t for d in deps)


def _compile(nvcc, src, obj, extra):
    cmd = [nvcc] + NVCC_FLAGS + extra + ["-c", src, "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    return src, r.returncode, r.stdout + r.stderr


def _marshal_stale(built_for):
    """Whether csrc/marshal.cpp is newer than its module, or that is of another PyTorch or Python."""
    src = os.path.join(CSRC, "marshal.cpp")
    if _stale(MARSHAL, [src, os.path.join(ROOT, "include", "w8lin.h"), os.path.abspath(__file__)]):
        return True
    try:
        with open(MARSHAL_FOR) as f:
            return f.read() != built_for
    except OSError:
        return True


def _marshal():
    """Compile the CPython module of csrc/marshal.cpp; returns what the compiler
    said where it failed (the binding then marshals in Python)."""
    import torch
    built_for = f"{torch.__version__} {sys.implementation.cache_tag}"
    if not _marshal_stale(built_for):
        return ""
    import sysconfig

    from torch.utils.cpp_extension import include_paths
    src = os.path.join(CSRC, "marshal.cpp")
    libs = os.path.join(os.path.dirname(torch.__file__), "lib")
    cuda = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(_nvcc()))), "include")
    tmp = f"{MARSHAL}.{os.getpid()}"
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-shared", f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}"]
    cmd += [f"-I{p}" for p in [*include_paths(), sysconfig.get_paths()["include"], cuda]]
    cmd += [f'-DW8_BUILT_FOR="{built_for}"', src, "-o", tmp, f"-L{libs}", "-ltorch_python", "-ltorch_cpu", "-lc10", "-lc10_cuda", f"-Wl,-rpath,{libs}"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode == 0:
        os.replace(tmp, MARSHAL)
        with open(MARSHAL_FOR, "w") as f:
            f.write(built_for)
        return ""
    return r.stdout + r.stderr


def build(verbose=False, extra_flags=()):
    """Compile and link; returns the path of the shared library."""
    nvcc = _nvcc()
    os.makedirs(OUT_DIR, exist_ok=True)
    hdrs = _headers()
    pool = cf.ThreadPoolExecutor(max_workers=1)
    marshal = pool.submit(_marshal)
    jobs = []
    objs = []
    for s in SOURCES:
        src = os.path.join(CSRC, s)
        obj = os.path.join(OUT_DIR, s.replace(".cu", ".o"))
        objs.append(obj)
        if _stale(obj, [src] + hdrs):
            jobs.append((src, obj))
    if jobs:
        with cf.ThreadPoolExecutor(max_workers=len(jobs)) as ex:
            futs = [ex.submit(_compile, nvcc, s, o, list(extra_flags)) for s, o in jobs]
            for f in futs:
                src, rc, out = f.result()
                if verbose and out.strip():
                    print(out, file=sys.stderr)
                if rc != 0:
                    raise RuntimeError(f"nvcc failed on {os.path.basename(src)}:\n{out}")
    if jobs or _stale(LIB, objs):
        cmd = [nvcc] + ARCH + ["-shared", "-o", LIB] + objs
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"link failed:\n{r.stdout}{r.stderr}")
    failed = marshal.result()
    pool.shutdown()
    if failed:
        print(f"csrc/marshal.cpp was not built; calls are marshalled in Python:\n{failed[-2000:]}", file=sys.stderr)
    return LIB


if __name__ == "__main__":
    print(build(verbose=True, extra_flags=sys.argv[1:]))
