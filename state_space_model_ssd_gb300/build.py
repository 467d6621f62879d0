"""Builds libssd.so (the CUDA kernels and the C ABI) in-tree for sm_103a, and the binding
of the operators around the scan to torch tensors.

Each .cu file is compiled by nvcc in parallel, then linked into
``state_space_model_ssd_gb300/libssd.so``; ``csrc/layer_ext.cpp`` is compiled beside them and
linked against it and torch's libraries into ``_layer_ext.so`` (left out where torch is not
installed).  No CMake.
"""

from __future__ import annotations

import concurrent.futures
import importlib.util
import os
import shutil
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
OBJDIR = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libssd.so")
EXT = os.path.join(PKG, "_layer_ext.so")
EXT_SRC = os.path.join(CSRC, "layer_ext.cpp")
LINKED = "layer_ext.linked"
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]


def _nvcc() -> str:
    cand = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(cand):
        raise RuntimeError("nvcc not found: the CUDA library cannot be built")
    return cand


def sources():
    return sorted(os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith(".cu"))


def _headers():
    hs = [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith((".cuh", ".h"))]
    hs += [os.path.join(INCLUDE, f) for f in os.listdir(INCLUDE) if f.endswith(".h")]
    return hs


def _ext_commands(cuda_home):
    """The compile command of the binding's object (which is of one torch version), the
    object, and its link command."""
    import torch
    root = os.path.dirname(os.path.abspath(torch.__file__))
    lib = os.path.join(root, "lib")
    obj = os.path.join(OBJDIR, "layer_ext-torch%s.o" % torch.__version__)
    cxx = shutil.which("g++") or "g++"
    compile_ = [cxx, "-std=c++17", "-O2", "-fPIC", "-fvisibility=hidden", "-I", INCLUDE,
                "-I", os.path.join(root, "include"),
                "-I", os.path.join(root, "include", "torch", "csrc", "api", "include"),
                "-I", sysconfig.get_paths()["include"], "-I", os.path.join(cuda_home, "include"),
                "-c", EXT_SRC, "-o", obj]
    link = [cxx, "-shared", obj, "-L", lib, "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_cuda",
            "-ltorch", "-ltorch_python", "-L", PKG, "-l:libssd.so", "-Wl,-rpath,$ORIGIN"]
    return compile_, obj, link


def _linked() -> str:
    """The object that _layer_ext.so was linked from."""
    try:
        with open(os.path.join(OBJDIR, LINKED)) as f:
            return f.read()
    except OSError:
        return ""


def _stale(target, deps) -> bool:
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(d) > t for d in deps)


def build(force: bool = False, verbose: bool = False) -> str:
    os.makedirs(OBJDIR, exist_ok=True)
    nvcc = _nvcc()
    hdrs = _headers()
    common = [nvcc, "-std=c++17", "-O3", "-lineinfo", *ARCH, "-Xcompiler", "-fPIC",
              "-I", INCLUDE, "-I", CSRC, "--expt-relaxed-constexpr"]
    if verbose:
        common += ["-Xptxas", "-v"]
    jobs = []
    objs = []
    for src in sources():
        obj = os.path.join(OBJDIR, os.path.basename(src)[:-3] + ".o")
        objs.append(obj)
        if force or _stale(obj, [src] + hdrs):
            jobs.append(common + ["-c", src, "-o", obj])
    # the binding alone needs torch: without it the C library is built all the same
    ext = None
    if importlib.util.find_spec("torch") is None:
        sys.stderr.write("torch is not installed: _layer_ext.so, the binding of the operators around the "
                         "scan, is not built\n")
    else:
        ext = _ext_commands(os.path.dirname(os.path.dirname(os.path.realpath(nvcc))))
    ext_jobs = [ext[0]] if ext and (force or _stale(ext[1], [EXT_SRC] + hdrs)) else []

    def failed(job, done):
        if verbose or done.returncode != 0:
            sys.stderr.write(done.stdout + done.stderr)
        if done.returncode == 0:
            return None
        return RuntimeError("%s failed on %s" % (os.path.basename(job[0]), job[job.index("-o") - 1]))

    errors, ext_errors = [], []
    if ext_jobs or jobs:
        with concurrent.futures.ThreadPoolExecutor(max_workers=min(16, len(ext_jobs + jobs))) as ex:
            futs = [ex.submit(subprocess.run, j, capture_output=True, text=True) for j in ext_jobs + jobs]
            for j, f in zip(ext_jobs + jobs, futs):
                (ext_errors if j in ext_jobs else errors).append(failed(j, f.result()))
    for e in filter(None, errors):
        raise e
    if force or jobs or _stale(LIB, objs):
        tmp = LIB + ".%d.tmp" % os.getpid()
        subprocess.run([nvcc, *ARCH, "-shared", "-cudart", "static", "-o", tmp, *objs],
                       check=True)
        os.replace(tmp, LIB)
    for e in filter(None, ext_errors):
        raise e
    # another torch's object may be older than the module linked since: the object linked is on record
    if ext and (force or _stale(EXT, [ext[1]]) or _linked() != os.path.basename(ext[1])):
        tmp = EXT + ".%d.tmp" % os.getpid()
        subprocess.run(ext[2] + ["-o", tmp], check=True)
        os.replace(tmp, EXT)
        with open(os.path.join(OBJDIR, LINKED), "w") as f:
            f.write(os.path.basename(ext[1]))
    return LIB


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose="-v" in sys.argv)
    print(LIB)
