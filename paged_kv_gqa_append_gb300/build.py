"""Build libpkv.so (the C-ABI library) in-tree with nvcc for sm_103a.

    python -m paged_kv_gqa_append_gb300.build [--force] [--ptxas-verbose]

Translation units compile in parallel; objects go to ``_build/`` at the repo
root and the shared library to ``paged_kv_gqa_append_gb300/libpkv.so``.
The CUDA runtime is linked statically, so the library loads on a machine
without a GPU driver (calls then fail with PKV_ERR_CUDA).  The Python binding's
marshalling of the small calls (binding/calls.cpp) is compiled against the
installed torch into ``paged_kv_gqa_append_gb300/_calls.so``, and again when that
is another one; libpkv.so itself needs neither Python's headers nor torch and is
built without them.
"""
from __future__ import annotations

import argparse
import concurrent.futures as cf
import importlib.metadata
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
BUILD = os.path.join(ROOT, "_build")
LIB = os.path.join(PKG, "libpkv.so")
BINDING = os.path.join(PKG, "binding", "calls.cpp")
BINDING_LIB = os.path.join(PKG, "_calls.so")

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
HOST_FLAGS = "-fPIC,-ffp-contract=off,-O2"
NVCC_FLAGS = ["-O3", "-std=c++17", "-lineinfo", *ARCH, "-Xcompiler", HOST_FLAGS,
              "-I", INCLUDE, "-I", CSRC]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libpkv.so")


def sources():
    return sorted(os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith((".cu", ".cpp")))


def _inputs():
    headers = [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith((".h", ".cuh"))]
    headers += [os.path.join(INCLUDE, f) for f in os.listdir(INCLUDE)]
    return sources() + headers + [os.path.abspath(__file__)]


def _older(target, inputs):
    return not os.path.exists(target) or any(os.path.getmtime(p) > os.path.getmtime(target) for p in inputs)


def _torch_dir():
    spec = importlib.util.find_spec("torch")
    return spec.submodule_search_locations[0] if spec is not None else None


def _stamp_path():
    return os.path.join(BUILD, "calls.torch")


def _torch_stamp() -> str:
    """What the binding is compiled against: torch, where it is, and Python."""
    try:
        version = importlib.metadata.version("torch")
    except importlib.metadata.PackageNotFoundError:
        version = "unknown"
    return f"torch {version} {_torch_dir()} python {sys.version_info.major}.{sys.version_info.minor}"


def binding_is_stale() -> bool:
    """Without torch there is no binding to build."""
    if _torch_dir() is None:
        return False
    if _older(BINDING_LIB, [BINDING, os.path.join(INCLUDE, "pkv.h"), os.path.abspath(__file__)]):
        return True
    try:
        with open(_stamp_path()) as f:
            return f.read() != _torch_stamp()
    except OSError:
        return True


def is_stale() -> bool:
    return _older(LIB, _inputs()) or binding_is_stale()


def _compile(src: str, ptxas_verbose: bool) -> tuple[str, str]:
    obj = os.path.join(BUILD, os.path.basename(src) + ".o")
    cmd = [nvcc(), *NVCC_FLAGS, "-c", src, "-o", obj]
    if ptxas_verbose and src.endswith(".cu"):
        cmd.append("-Xptxas=-v")
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc failed for {os.path.basename(src)}:\n{r.stdout}\n{r.stderr}")
    return obj, r.stderr


def _compile_binding() -> str:
    obj = os.path.join(BUILD, "calls.cpp.o")
    torch = _torch_dir()
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(nvcc())))
    cmd = [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-fvisibility=hidden", "-c", BINDING, "-o", obj,
           "-I", INCLUDE, "-isystem", os.path.join(torch, "include"),
           "-isystem", os.path.join(torch, "include", "torch", "csrc", "api", "include"),
           "-isystem", sysconfig.get_paths()["include"], "-isystem", os.path.join(cuda, "include")]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"{cmd[0]} failed for calls.cpp:\n{r.stdout}\n{r.stderr}")
    return obj


def _link_binding(obj: str):
    torch = _torch_dir()
    tmp = BINDING_LIB + ".tmp"
    cmd = [os.environ.get("CXX", "g++"), "-shared", "-o", tmp, obj, "-L", PKG, "-lpkv", "-Wl,-rpath,$ORIGIN",
           "-L", os.path.join(torch, "lib"), "-ltorch_python", "-ltorch_cpu", "-lc10_cuda", "-lc10"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link of _calls.so failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, BINDING_LIB)
    with open(_stamp_path(), "w") as f:
        f.write(_torch_stamp())


def build(force: bool = False, ptxas_verbose: bool = False, quiet: bool = True) -> str:
    """Compile every translation unit and link libpkv.so; returns its path."""
    if not force and not ptxas_verbose and not is_stale():
        return LIB
    os.makedirs(BUILD, exist_ok=True)
    whole = force or ptxas_verbose or _older(LIB, _inputs())
    srcs = sources() if whole else []
    with cf.ThreadPoolExecutor(max_workers=min(12, len(srcs) + 1)) as ex:
        binding = ex.submit(_compile_binding) if _torch_dir() is not None else None
        results = list(ex.map(lambda s: _compile(s, ptxas_verbose), srcs))
    logs = "".join(e for _, e in results)
    if ptxas_verbose:
        with open(os.path.join(BUILD, "ptxas.log"), "w") as f:
            f.write(logs)
    if whole:
        tmp = LIB + ".tmp"
        cmd = [nvcc(), *ARCH, "-shared", "-cudart", "static", "-o", tmp, *[o for o, _ in results]]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
        os.replace(tmp, LIB)
    if binding is not None:  # what may be wrong with it does not keep the library from being built
        _link_binding(binding.result())
    if not quiet:
        print(f"built {LIB}" + ("" if binding is not None else " (without the Python binding's _calls.so: no torch)"))
        if ptxas_verbose:
            print(logs)
    return LIB


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__)
    ap.add_argument("--force", action="store_true")
    ap.add_argument("--ptxas-verbose", action="store_true")
    a = ap.parse_args(argv)
    build(force=a.force, ptxas_verbose=a.ptxas_verbose, quiet=False)


if __name__ == "__main__":
    sys.exit(main())
