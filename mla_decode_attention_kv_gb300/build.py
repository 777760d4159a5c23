"""Build the CUDA library ``libmla_dcp.so`` in-tree with nvcc for sm_103a, and
``_native.so``, the Python binding of its cache operators, with g++ against
the installed PyTorch.

Each translation unit is compiled in parallel, then linked into the shared
libraries next to this file.  A stamp of the sources and flags skips rebuilds
when nothing changed.
"""
from __future__ import annotations

import hashlib
import importlib.util
import os
import shutil
import subprocess
import sysconfig
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(os.path.dirname(HERE), "include")
LIB_PATH = os.path.join(HERE, "libmla_dcp.so")
NATIVE_PATH = os.path.join(HERE, "_native.so")
BUILD_DIR = os.path.join(HERE, "_build")
SOURCES = ["api.cu", "partial.cu", "partial_fp8.cu", "combine_vup.cu", "gather.cu",
           "partial_fp4.cu", "append.cu", "pages.cu"]
NATIVE_SOURCE = "bindings.cpp"
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ARCH + ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC",
                     "-I" + INCLUDE]


def _nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libmla_dcp.so")


def _torch_dir() -> str:
    """The installed torch package (found without importing it)."""
    spec = importlib.util.find_spec("torch")
    if spec is None or not spec.submodule_search_locations:
        raise RuntimeError("PyTorch is required to build the Python binding")
    return list(spec.submodule_search_locations)[0]


def _native_flags() -> list:
    inc = os.path.join(_torch_dir(), "include")
    cuda = os.path.join(os.path.dirname(os.path.dirname(_nvcc())), "include")
    dirs = [inc, os.path.join(inc, "torch", "csrc", "api", "include"),
            sysconfig.get_paths()["include"], cuda]
    return ["-O2", "-std=c++17", "-fPIC", "-w"] + [x for d in dirs for x in ("-isystem", d)]


def _stamp() -> str:
    h = hashlib.sha256()
    h.update(" ".join(NVCC_FLAGS + _native_flags()).encode())
    with open(os.path.join(_torch_dir(), "version.py"), "rb") as f:
        h.update(f.read())
    for d in (CSRC, INCLUDE):
        for name in sorted(os.listdir(d)):
            if name.endswith((".cu", ".cuh", ".cpp", ".h")):
                with open(os.path.join(d, name), "rb") as f:
                    h.update(name.encode())
                    h.update(f.read())
    return h.hexdigest()


def build(force: bool = False, verbose: bool = False) -> str:
    """Compile (if needed) and return the path of libmla_dcp.so."""
    stamp_path = LIB_PATH + ".stamp"
    stamp = _stamp()
    if (not force and os.path.exists(LIB_PATH) and os.path.exists(NATIVE_PATH)
            and os.path.exists(stamp_path)
            and open(stamp_path).read() == stamp):
        return LIB_PATH
    nvcc = _nvcc()
    os.makedirs(BUILD_DIR, exist_ok=True)

    def compile_one(src: str) -> str:
        obj = os.path.join(BUILD_DIR, os.path.splitext(src)[0] + ".o")
        if src.endswith(".cpp"):
            cmd = ["g++", *_native_flags(), "-c", os.path.join(CSRC, src), "-o", obj]
        else:
            cmd = [nvcc, *NVCC_FLAGS, "-c", os.path.join(CSRC, src), "-o", obj]
            if verbose:
                cmd.insert(1, "-Xptxas=-v")
        res = subprocess.run(cmd, capture_output=True, text=True)
        if res.returncode != 0:
            raise RuntimeError(f"{cmd[0]} failed on {src}:\n{res.stderr}")
        if verbose and res.stderr:
            print(res.stderr)
        return obj

    with ThreadPoolExecutor(max_workers=len(SOURCES) + 1) as ex:
        *objs, native = ex.map(compile_one, SOURCES + [NATIVE_SOURCE])

    def link(cmd: list, path: str) -> None:
        res = subprocess.run([*cmd, "-o", path + ".tmp"], capture_output=True, text=True)
        if res.returncode != 0:
            raise RuntimeError(f"link of {os.path.basename(path)} failed:\n{res.stderr}")
        os.replace(path + ".tmp", path)

    link([nvcc, *ARCH, "-shared", *objs], LIB_PATH)
    # (PyTorch's libraries are in the process once torch is imported)
    libs = ["torch_python", "torch", "torch_cpu", "torch_cuda", "c10", "c10_cuda"]
    link(["g++", "-shared", native, "-L" + os.path.join(_torch_dir(), "lib"),
          "-Wl,--no-as-needed", *("-l" + x for x in libs), "-L" + HERE, "-l:libmla_dcp.so",
          "-Wl,-rpath,$ORIGIN"], NATIVE_PATH)
    with open(stamp_path, "w") as f:
        f.write(stamp)
    return LIB_PATH


if __name__ == "__main__":
    print(build(force=True, verbose=True))
