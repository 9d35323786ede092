"""Builds libindexer_bwd.so in-tree with nvcc for sm_103a, and the Python
marshalling of the training operators (_train.so) with g++.

Each .cu translation unit compiles in parallel to an object, then nvcc links
the shared library (CUDA runtime linked statically, plain C ABI); _train.so is
linked against it and torch's libraries.
"""
from __future__ import annotations

import glob
import os
import shutil
import subprocess
import tempfile

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(PKG, "libindexer_bwd.so")
TRAIN = os.path.join(PKG, "_train.so")
TRAIN_SOURCES = [os.path.join(CSRC, name) for name in ("train_binding.cpp", "heads_binding.cpp")]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-Xcompiler", "-fvisibility=hidden",
         "--expt-relaxed-constexpr"]


def _sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _inputs():
    return _sources() + TRAIN_SOURCES + glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(CSRC, "*.h")) + \
        glob.glob(os.path.join(INCLUDE, "*.h"))


def nvcc() -> str:
    for cand in (shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libindexer_bwd.so")


def _train_flags():
    """Compiler and linker flags of _train.so: Python's, torch's and CUDA's headers and libraries."""
    import sysconfig

    import torch
    root = os.path.dirname(torch.__file__)
    cuda = os.path.dirname(os.path.dirname(nvcc()))
    include = [sysconfig.get_paths()["include"], os.path.join(root, "include"),
               os.path.join(root, "include", "torch", "csrc", "api", "include"), os.path.join(cuda, "include"), INCLUDE]
    compile_ = ["-O2", "-std=c++17", "-fPIC", "-fvisibility=hidden", "-w",
                f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}"]
    for d in include:
        compile_ += ["-isystem" if d != INCLUDE else "-I", d]
    link = ["-shared", f"-L{os.path.join(root, 'lib')}", f"-Wl,-rpath,{os.path.join(root, 'lib')}", "-Wl,-rpath,$ORIGIN",
            "-ltorch_python", "-ltorch", "-ltorch_cpu", "-ltorch_cuda", "-lc10", "-lc10_cuda"]
    return compile_, link


def stale() -> bool:
    if not os.path.exists(LIB) or not os.path.exists(TRAIN):
        return True
    t = min(os.path.getmtime(LIB), os.path.getmtime(TRAIN))
    return any(os.path.getmtime(f) > t for f in _inputs())


def build(force: bool = False, verbose: bool = False) -> str:
    if not force and not stale():
        return LIB
    cc = nvcc()
    with tempfile.TemporaryDirectory(prefix="ibwd_build_") as tmp:
        procs = []
        objs = []
        for src in _sources():
            obj = os.path.join(tmp, os.path.basename(src) + ".o")
            cmd = [cc, *ARCH, *FLAGS, "-I", INCLUDE, "-c", src, "-o", obj]
            if verbose:
                cmd.insert(1, "-Xptxas=-v")
            procs.append((src, subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT)))
            objs.append(obj)
        compile_, link = _train_flags()
        train_objs = []
        for src in TRAIN_SOURCES:
            train_objs.append(os.path.join(tmp, os.path.basename(src) + ".o"))
            procs.append((src, subprocess.Popen(["g++", *compile_, "-c", src, "-o", train_objs[-1]],
                                                stdout=subprocess.PIPE, stderr=subprocess.STDOUT)))
        errs = []
        for src, pr in procs:
            out, _ = pr.communicate()
            if pr.returncode != 0:
                errs.append(f"{src}:\n{out.decode(errors='replace')}")
            elif verbose and out:
                print(out.decode(errors="replace"))
        if errs:
            raise RuntimeError("compilation failed:\n" + "\n".join(errs))
        tmp_lib = os.path.join(tmp, "libindexer_bwd.so")
        subprocess.check_call([cc, *ARCH, "-shared", *objs, "-o", tmp_lib])
        shutil.copyfile(tmp_lib, LIB + f".tmp{os.getpid()}")
        os.replace(LIB + f".tmp{os.getpid()}", LIB)
        tmp_train = TRAIN + f".tmp{os.getpid()}"
        subprocess.check_call(["g++", *train_objs, "-o", tmp_train, f"-L{PKG}", "-l:libindexer_bwd.so", *link])
        os.replace(tmp_train, TRAIN)
    return LIB


if __name__ == "__main__":
    import sys
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
