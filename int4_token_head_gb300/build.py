"""Build libkvint4.so in-tree with nvcc for sm_103a (GB300).

The translation units are compiled in parallel and linked with the static
CUDA runtime, so loading the library needs only the NVIDIA driver.  A stamp
file records the host architecture and a hash of the sources, so a library
built on another machine (or from other sources) is rebuilt.  The Python call
module of the FP8 operators, named for its interpreter, is built beside it and
again whenever it is missing.
"""

from __future__ import annotations

import hashlib
import importlib.util
import os
import platform
import shutil
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
BUILD_DIR = os.path.join(PKG, "_build")
LIB_PATH = os.path.join(PKG, "libkvint4.so")
STAMP = os.path.join(BUILD_DIR, "stamp.txt")
HEADER = os.path.join(ROOT, "include", "kvint4.h")

SOURCES = ["api.cu", "write.cu", "write_int8.cu", "attention.cu", "rht.cu", "attention_fp8.cu", "attention_shared_fp8.cu",
           "cache_fp8.cu", "evict_fp8.cu", "mass_fp8.cu", "norm_rope.cu", "api_fp8.cu", "timing.cu", "noalloc.cu", "selftest.cu"]
BINDING_SRC = os.path.join(CSRC, "fp8_binding.cpp")
PYTHON_TAG = sysconfig.get_config_var("EXT_SUFFIX") or ".so"  # the interpreter's own: another one does not import it
BINDING_PATH = os.path.join(PKG, "_fp8_binding" + PYTHON_TAG)
GENCODE = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "-Xcompiler", "-fvisibility=hidden"]


def nvcc_path() -> str:
    cand = shutil.which("nvcc")
    if cand:
        return cand
    for p in ("/usr/local/cuda/bin/nvcc",):
        if os.path.exists(p):
            return p
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libkvint4.so")


def _inputs():
    files = [os.path.join(CSRC, f) for f in sorted(os.listdir(CSRC))
             if f.endswith((".cu", ".cuh", ".h", ".cpp"))]
    return files + [HEADER, os.path.abspath(__file__)]


def _torch_dir():
    spec = importlib.util.find_spec("torch")
    return spec.submodule_search_locations[0] if spec else None


def _binding_command():
    """g++ for the Python call module, which sees torch's tensors; None where it
    cannot be built: without g++, Python's headers or a torch with CUDA."""
    torch, py = _torch_dir(), sysconfig.get_paths()["include"]
    if torch is None or not os.path.exists(os.path.join(py, "Python.h")) or shutil.which("g++") is None:
        return None
    lib = os.path.join(torch, "lib")
    if not os.path.exists(os.path.join(lib, "libc10_cuda.so")):
        return None
    cuda = os.path.join(os.path.dirname(os.path.dirname(nvcc_path())), "include")
    return ["g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden", "-I", os.path.join(torch, "include"),
            "-I", os.path.join(torch, "include", "torch", "csrc", "api", "include"), "-I", py, "-I", cuda, BINDING_SRC,
            "-o", BINDING_PATH + ".tmp", "-L", lib, "-ltorch_python", "-ltorch_cpu", "-lc10", "-lc10_cuda"]


def _fingerprint(extra=()) -> str:
    h = hashlib.sha256()
    h.update(platform.machine().encode())
    h.update(PYTHON_TAG.encode())
    torch = _torch_dir()
    if torch:  # the call module depends on its version
        with open(os.path.join(torch, "version.py"), "rb") as fh:
            h.update(fh.read())
    for f in _inputs():
        with open(f, "rb") as fh:
            h.update(os.path.basename(f).encode())
            h.update(fh.read())
    for e in extra:
        h.update(str(e).encode())
    return h.hexdigest()


def _library_is_current(extra=()) -> bool:
    if not os.path.exists(LIB_PATH) or not os.path.exists(STAMP):
        return False
    with open(STAMP) as f:
        return f.read().strip() == _fingerprint(extra)


def is_current(extra=()) -> bool:
    return _library_is_current(extra) and (os.path.exists(BINDING_PATH) or _binding_command() is None)


def _start_binding():
    """Starts building the call module; what was there goes first."""
    for old in (BINDING_PATH, os.path.join(PKG, "_fp8_binding.so")):
        if os.path.exists(old):
            os.remove(old)
    cmd = _binding_command()
    return cmd and subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True)


def _finish_binding(proc):
    if proc is None:  # it cannot be built here: the same calls go through ctypes, some microseconds slower
        return
    out, _ = proc.communicate()
    if proc.returncode != 0:
        raise RuntimeError(f"g++ failed for {os.path.basename(BINDING_SRC)}:\n{out}")
    os.replace(BINDING_PATH + ".tmp", BINDING_PATH)


def build(force: bool = False, verbose: bool = False, ptxas_info: bool = False) -> str:
    """Compile (if needed) and return the path of libkvint4.so."""
    if not force and is_current():
        return LIB_PATH
    if not force and _library_is_current():  # the call module alone is missing
        _finish_binding(_start_binding())
        return LIB_PATH
    nvcc = nvcc_path()
    os.makedirs(BUILD_DIR, exist_ok=True)
    procs = []
    objs = []
    for src in SOURCES:
        obj = os.path.join(BUILD_DIR, src.replace(".cu", ".o"))
        objs.append(obj)
        cmd = [nvcc, *GENCODE, *NVCC_FLAGS, "-c", os.path.join(CSRC, src), "-o", obj]
        if ptxas_info:
            cmd.insert(1, "-Xptxas=-v")
        if verbose:
            print(" ".join(cmd), file=sys.stderr)
        procs.append((src, subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True)))
    binding = _start_binding()
    logs = {}
    failed = []
    for src, p in procs:
        out, _ = p.communicate()
        logs[src] = out
        if p.returncode != 0:
            failed.append(src)
    _finish_binding(binding)
    if failed:
        msg = "\n".join(f"--- {s} ---\n{logs[s]}" for s in failed)
        raise RuntimeError(f"nvcc failed for {failed}:\n{msg}")
    tmp = LIB_PATH + ".tmp"
    link = [nvcc, *GENCODE, "-shared", "-cudart", "static", "-o", tmp, *objs]
    r = subprocess.run(link, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}")
    os.replace(tmp, LIB_PATH)
    with open(STAMP, "w") as f:
        f.write(_fingerprint())
    if verbose or ptxas_info:
        for s in SOURCES:
            if logs[s].strip():
                print(f"--- {s} ---\n{logs[s]}", file=sys.stderr)
    return LIB_PATH


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose=True, ptxas_info="--ptxas" in sys.argv)
    print(LIB_PATH)
