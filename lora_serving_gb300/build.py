"""Builds ``liblora.so`` (the C-ABI CUDA library) in-tree with nvcc for sm_103a, and
``_pycalls.so``, the Python side of some of its calls, with gcc.

Each translation unit compiles in parallel into ``_build/``; the shared
library lands next to this file.  No cmake, one ``-gencode``.
"""
from __future__ import annotations

import concurrent.futures as cf
import os
import shutil
import subprocess
import sys
import sysconfig
import warnings

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(HERE, "liblora.so")
CALLS = os.path.join(HERE, "_pycalls.so")

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]


def _cuda_home() -> str:
    home = os.environ.get("CUDA_HOME") or os.environ.get("CUDA_PATH")
    if home and os.path.exists(os.path.join(home, "bin", "nvcc")):
        return home
    nvcc = shutil.which("nvcc")
    if nvcc:
        return os.path.dirname(os.path.dirname(os.path.realpath(nvcc)))
    return "/usr/local/cuda"


def _sources():
    return sorted(f for f in os.listdir(CSRC) if f.endswith((".cu", ".cpp")))


def _stale(out, names) -> bool:
    """Whether `out` is missing or older than one of these files of csrc/, or the header."""
    if not os.path.exists(out):
        return True
    deps = [os.path.join(CSRC, f) for f in names] + [os.path.join(INCLUDE, "lora.h")]
    return any(os.path.getmtime(p) > os.path.getmtime(out) for p in deps)


def build(force: bool = False, verbose: bool = False, extra_flags=()) -> str:
    """Compile every source under csrc/ and link liblora.so; returns its path.
    Then _pycalls.so, without which the calls that need it raise: on a machine
    that lacks a C compiler or Python's headers there is a warning here."""
    if force or _stale(LIB, [f for f in os.listdir(CSRC) if f != "pycalls.c"]):
        _build_lib(verbose, extra_flags)
    if force or _stale(CALLS, ["pycalls.c"]):
        try:
            _build_calls()
        except (OSError, RuntimeError) as e:
            if os.path.exists(CALLS):   # of another version of the library
                os.remove(CALLS)
            warnings.warn(f"no {os.path.basename(CALLS)}: lora_rms_norm and lora_kv4_* cannot be called from Python ({e})")
    return LIB


def _build_lib(verbose, extra_flags):
    cuda = _cuda_home()
    nvcc = os.path.join(cuda, "bin", "nvcc")
    os.makedirs(BUILD, exist_ok=True)
    common = ["-std=c++17", "-O3", "-I", INCLUDE, "-I", CSRC, "-Xcompiler", "-fPIC"]

    def compile_one(src):
        obj = os.path.join(BUILD, src + ".o")
        path = os.path.join(CSRC, src)
        if src.endswith(".cu"):
            cmd = [nvcc, *ARCH, "-lineinfo", *common, "-Xptxas", "-warn-spills", *extra_flags,
                   "-c", path, "-o", obj]
        else:
            cmd = [nvcc, *common, "-Xcompiler", "-Wall", "-c", path, "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {src}:\n{' '.join(cmd)}\n{r.stdout}\n{r.stderr}")
        if verbose and (r.stdout or r.stderr):
            sys.stderr.write(r.stdout + r.stderr)
        return obj

    srcs = _sources()
    with cf.ThreadPoolExecutor(max_workers=min(8, len(srcs))) as ex:
        objs = list(ex.map(compile_one, srcs))
    tmp = LIB + f".tmp{os.getpid()}"
    lib_dir = os.path.join(cuda, "lib64")
    cmd = [nvcc, *ARCH, "-shared", "-cudart", "shared", "-o", tmp, *objs,
           "-Xlinker", f"-rpath,{lib_dir}"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{' '.join(cmd)}\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)


def _build_calls():
    """The Python side of some calls: plain C against the interpreter's headers (abi.py hands it the library's functions)."""
    tmp = CALLS + f".tmp{os.getpid()}"
    cmd = [os.environ.get("CC", "gcc"), "-O2", "-Wall", "-fPIC", "-shared", "-I", sysconfig.get_paths()["include"], "-I", INCLUDE,
           os.path.join(CSRC, "pycalls.c"), "-o", tmp]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"gcc failed on pycalls.c:\n{' '.join(cmd)}\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, CALLS)


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True))
