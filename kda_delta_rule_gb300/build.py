"""Build the KDA CUDA library in-tree: kda_delta_rule_gb300/libkda.so.

Each translation unit under csrc/ is compiled by nvcc for sm_103a in
parallel, then linked into one shared library against the shared CUDA
runtime (libcudart.so.13).  Inside a PyTorch process the loader reuses the
runtime PyTorch already loaded, so both see the same current device; outside
one, the rpath finds the toolkit's copy.  kda_delta_rule_gb300/_kda_torch.so, the
native part of the Python binding, is compiled beside it by the host compiler
against PyTorch's headers and linked to libkda.so.

    python -m kda_delta_rule_gb300.build [--force] [-j N]
"""
from __future__ import annotations

import argparse
import importlib.util
import os
import shutil
import subprocess
import sys
import sysconfig
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libkda.so")
BINDING = os.path.join(PKG, "binding", "kda_torch.cpp")
BINDING_LIB = os.path.join(PKG, "_kda_torch.so")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
COMMON = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "-I", os.path.join(ROOT, "include")]


def _nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the KDA library needs the CUDA 13 toolkit")


def _cxx() -> str:
    for cand in (os.environ.get("CXX"), "g++", "c++"):
        if cand and shutil.which(cand):
            return cand
    raise RuntimeError("no C++ compiler found for the Python binding")


def sources():
    return sorted(os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith((".cu", ".cpp")))


def _deps_mtime():
    files = [os.path.join(CSRC, f) for f in os.listdir(CSRC)]
    files.append(os.path.join(ROOT, "include", "kda.h"))
    files += [os.path.abspath(__file__), BINDING]
    return max(os.path.getmtime(f) for f in files)


def build(force: bool = False, jobs: int | None = None, verbose: bool = False) -> str:
    newest = _deps_mtime()
    if not force and all(os.path.exists(f) and os.path.getmtime(f) >= newest for f in (LIB, BINDING_LIB)):
        return LIB
    nvcc = _nvcc()
    os.makedirs(BUILD, exist_ok=True)
    srcs = sources()

    def compile_one(src):
        obj = os.path.join(BUILD, os.path.basename(src) + ".o")
        cmd = [nvcc, *ARCH, *COMMON, "-c", src, "-o", obj]
        if verbose:
            cmd.insert(1, "-Xptxas=-v")
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {os.path.basename(src)}:\n{r.stdout}\n{r.stderr}")
        return obj, r.stderr

    torch_dir = os.path.dirname(importlib.util.find_spec("torch").origin)
    binding_obj = os.path.join(BUILD, "kda_torch.o")

    def compile_binding():
        include = [os.path.join(torch_dir, "include"), sysconfig.get_paths()["include"],
                   os.path.join(os.path.dirname(os.path.dirname(nvcc)), "include")]
        cmd = [_cxx(), "-O2", "-std=c++17", "-fPIC", *(f"-I{d}" for d in include), "-c", BINDING, "-o", binding_obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"{cmd[0]} failed on {os.path.basename(BINDING)}:\n{r.stdout}\n{r.stderr}")

    with ThreadPoolExecutor(max_workers=jobs or min(8, os.cpu_count() or 4)) as ex:
        binding = ex.submit(compile_binding)
        results = list(ex.map(compile_one, srcs))
        binding.result()
    objs = [o for o, _ in results]
    if verbose:
        for _, log in results:
            sys.stderr.write(log)
    tmp = LIB + ".tmp"
    cudalib = os.path.join(os.path.dirname(os.path.dirname(nvcc)), "lib64")
    cmd = [nvcc, *ARCH, "-shared", "-cudart", "shared", f"-Xlinker=-rpath,{cudalib}", "-o", tmp, *objs]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)
    tmp = BINDING_LIB + ".tmp"
    torch_lib = os.path.join(torch_dir, "lib")
    cmd = [_cxx(), "-shared", "-o", tmp, binding_obj, "-L", PKG, "-l:libkda.so", "-L", torch_lib, "-lc10", "-lc10_cuda",
           "-ltorch_cpu", "-ltorch_cuda", "-ltorch_python", "-Wl,-rpath,$ORIGIN", f"-Wl,-rpath,{torch_lib}"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link of the binding failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, BINDING_LIB)
    return LIB


if __name__ == "__main__":
    ap = argparse.ArgumentParser()
    ap.add_argument("--force", action="store_true")
    ap.add_argument("-j", type=int, default=None)
    ap.add_argument("-v", action="store_true")
    args = ap.parse_args()
    print(build(force=args.force, jobs=args.j, verbose=args.v))
