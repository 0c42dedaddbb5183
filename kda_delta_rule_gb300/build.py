"""Build the KDA CUDA library in-tree: kda_delta_rule_gb300/libkda.so.

Each translation unit under csrc/ is compiled by nvcc for sm_103a in
parallel, then linked into one shared library against the shared CUDA
runtime (libcudart.so.13).  Inside a PyTorch process the loader reuses the
runtime PyTorch already loaded, so both see the same current device; outside
one, the rpath finds the toolkit's copy.  kda_delta_rule_gb300/_kda_torch.so, the
native part of the Python binding, is compiled beside it by the host compiler
against PyTorch's headers and linked to libkda.so.
It is remade for another PyTorch or Python; where it cannot be made, kda.py does
without.

    python -m kda_delta_rule_gb300.build [--force] [-j N]
"""
from __future__ import annotations

import argparse
import importlib.util
import os
import re
import shutil
import subprocess
import sys
import sysconfig
import warnings
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libkda.so")
BINDING = os.path.join(PKG, "binding", "kda_torch.cpp")
BINDING_LIB = os.path.join(PKG, "_kda_torch.so")
BINDING_FOR = os.path.join(PKG, "_kda_torch.made_for")
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


def _fresh(lib, files):
    return os.path.exists(lib) and os.path.getmtime(lib) >= max(os.path.getmtime(f) for f in files)


def this_torch() -> str:
    """The PyTorch and the Python that the binding's native part has to be made for."""
    spec = importlib.util.find_spec("torch")
    version = None
    if spec is not None:
        with open(os.path.join(os.path.dirname(spec.origin), "version.py")) as f:
            version = re.search(r"__version__\s*=\s*['\"](.+?)['\"]", f.read())
    return f"torch {version.group(1) if version else None}, {sysconfig.get_config_var('SOABI')}"


def binding_made_for() -> str:
    """The same of the native part that is there ("" if that is not known)."""
    if not os.path.exists(BINDING_FOR):
        return ""
    with open(BINDING_FOR) as f:
        return f.read().strip()


def _build_binding(nvcc):
    """Compile the native part of the Python binding; returns its object file."""
    torch_spec = importlib.util.find_spec("torch")
    if torch_spec is None:
        raise RuntimeError("PyTorch not found: the Python binding is built against it")
    torch_dir = os.path.dirname(torch_spec.origin)
    obj = os.path.join(BUILD, "kda_torch.o")
    include = [os.path.join(torch_dir, "include"), sysconfig.get_paths()["include"],
               os.path.join(os.path.dirname(os.path.dirname(nvcc)), "include")]
    _run([_cxx(), "-O2", "-std=c++17", "-fPIC", *(f"-I{d}" for d in include), "-c", BINDING, "-o", obj],
         os.path.basename(BINDING))
    return obj, os.path.join(torch_dir, "lib")


def _link_binding(obj, torch_lib):
    tmp = BINDING_LIB + ".tmp"
    _run([_cxx(), "-shared", "-o", tmp, obj, "-L", PKG, "-l:libkda.so", "-L", torch_lib, "-lc10", "-lc10_cuda",
          "-ltorch_cpu", "-ltorch_cuda", "-ltorch_python", "-Wl,-rpath,$ORIGIN", f"-Wl,-rpath,{torch_lib}"], "the binding's link")
    os.replace(tmp, BINDING_LIB)
    with open(BINDING_FOR, "w") as f:
        f.write(this_torch() + "\n")


def _run(cmd, what):
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"{os.path.basename(cmd[0])} failed on {what}:\n{r.stdout}\n{r.stderr}")
    return r.stderr


def build(force: bool = False, jobs: int | None = None, verbose: bool = False) -> str:
    """Build what is older than its sources.  The library has to build; without the binding's native part (no Python or
    PyTorch headers, say) a warning is given, and kda.py makes its calls through ctypes."""
    shared = [os.path.join(ROOT, "include", "kda.h"), os.path.abspath(__file__)]
    csrc = [os.path.join(CSRC, f) for f in os.listdir(CSRC)]
    lib_stale = force or not _fresh(LIB, csrc + shared)
    binding_stale = force or lib_stale or not _fresh(BINDING_LIB, [BINDING, *shared]) or binding_made_for() != this_torch()
    if not (lib_stale or binding_stale):
        return LIB
    nvcc = _nvcc()
    os.makedirs(BUILD, exist_ok=True)

    def compile_one(src):
        obj = os.path.join(BUILD, os.path.basename(src) + ".o")
        cmd = [nvcc, *ARCH, *COMMON, "-c", src, "-o", obj]
        if verbose:
            cmd.insert(1, "-Xptxas=-v")
        return obj, _run(cmd, os.path.basename(src))

    with ThreadPoolExecutor(max_workers=jobs or min(8, os.cpu_count() or 4)) as ex:
        binding = ex.submit(_build_binding, nvcc)
        results = list(ex.map(compile_one, sources() if lib_stale else []))
    if lib_stale:
        if verbose:
            for _, log in results:
                sys.stderr.write(log)
        tmp = LIB + ".tmp"
        cudalib = os.path.join(os.path.dirname(os.path.dirname(nvcc)), "lib64")
        _run([nvcc, *ARCH, "-shared", "-cudart", "shared", f"-Xlinker=-rpath,{cudalib}", "-o", tmp, *(o for o, _ in results)],
             "the library's link")
        os.replace(tmp, LIB)
    try:
        _link_binding(*binding.result())
    except RuntimeError as e:
        if os.path.exists(BINDING_LIB):
            os.remove(BINDING_LIB)              # made for another state of the library
        warnings.warn(f"the native part of the Python binding was not built; calls go through ctypes\n{e}", RuntimeWarning)
    return LIB


if __name__ == "__main__":
    ap = argparse.ArgumentParser()
    ap.add_argument("--force", action="store_true")
    ap.add_argument("-j", type=int, default=None)
    ap.add_argument("-v", action="store_true")
    args = ap.parse_args()
    print(build(force=args.force, jobs=args.j, verbose=args.v))
