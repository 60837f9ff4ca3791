"""Build the CUDA library ``csr_spmm_gb300/lib/libcsrspmm.so`` for sm_103a.

Each translation unit under ``csrc/`` is compiled by its own nvcc process
(in parallel), then the objects are linked into one shared library on the shared
CUDA runtime.  Beside it g++ builds two Python modules for short calls: ``_lm_calls.so``
calls the language-model entry points, ``_torch_outputs.so`` makes the torch wrappers'
output tensors.  The library needs nvcc alone: a module is left out where Python's headers or
a CUDA build of torch are missing, and one that fails is reported when the library is in place.
A rebuild happens only when a source, header or flag changed (a content hash is kept
beside the library).

Run ``python -m csr_spmm_gb300.build`` or call :func:`build`.
"""
from __future__ import annotations

import hashlib
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
INCLUDE = os.path.join(ROOT, "include")
OBJ_DIR = os.path.join(PKG, "_build")
LIB_DIR = os.path.join(PKG, "lib")
LIB = os.path.join(LIB_DIR, "libcsrspmm.so")

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ARCH + ["-O3", "-lineinfo", "-std=c++20", "-Xcompiler", "-fPIC",
                     "--expt-relaxed-constexpr", "-I", INCLUDE, "-I", CSRC]
# The CUDA runtime is the process's shared one.  A second, static one costs 2.3 us (of 12)
# in each small call between torch's own: a lookup that makes its output takes 9.6 us.
LINK_FLAGS = ["-shared", "--cudart", "shared"]


def _nvcc() -> str:
    for cand in (shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA 13 toolkit is required to build csr_spmm_gb300")


def _runtime_path(nvcc: str) -> list:
    """Where the library finds libcudart when no one in the process has loaded it."""
    lib = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(nvcc))), "lib64")
    return ["-Xlinker", "-rpath," + lib] if os.path.isdir(lib) else []


def _left_out(name: str, why: str) -> None:
    sys.stderr.write(f"csr_spmm_gb300.build: _{name} is left out ({why}); the language-model "
                     "wrappers need it, the library does not\n")


def _module(name: str, deps, flags, libs, force: bool) -> None:
    """Build csrc/<name>.cpp, a Python module, with the host compiler."""
    src, out = os.path.join(CSRC, name + ".cpp"), os.path.join(LIB_DIR, "_" + name + ".so")
    if not os.path.exists(os.path.join(sysconfig.get_paths()["include"], "Python.h")):
        return _left_out(name, "no Python.h")
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-shared", src, "-I", INCLUDE,
           "-isystem", sysconfig.get_paths()["include"]] + flags + libs
    h = hashlib.sha256(" ".join(cmd).encode())
    for dep in [src] + deps:
        with open(dep, "rb") as f:
            h.update(f.read())
    stamp = out + ".sha256"
    if not force and os.path.exists(out) and os.path.exists(stamp):
        with open(stamp) as f:
            if f.read().strip() == h.hexdigest():
                return
    os.makedirs(LIB_DIR, exist_ok=True)
    tmp = out + f".tmp{os.getpid()}"
    r = subprocess.run(cmd + ["-o", tmp], capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed on {name}.cpp:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, out)
    with open(stamp, "w") as f:
        f.write(h.hexdigest() + "\n")


def _lm_calls(force: bool = False) -> None:
    """The module that calls the language-model entry points."""
    _module("lm_calls", [os.path.join(INCLUDE, "csr_spmm.h")], [], [], force)


def _torch_outputs(force: bool = False) -> None:
    """The module that makes the torch wrappers' outputs (none without torch for CUDA)."""
    spec = importlib.util.find_spec("torch")
    if spec is None:
        return
    torch = list(spec.submodule_search_locations)[0]
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(_nvcc())))
    libs = os.path.join(torch, "lib")
    if not os.path.exists(os.path.join(libs, "libtorch_cuda.so")):
        return _left_out("torch_outputs", "torch is built without CUDA")
    _module("torch_outputs", [os.path.join(torch, "version.py")],
            ["-isystem", os.path.join(torch, "include"), "-isystem", os.path.join(cuda, "include")],
            ["-L" + libs, "-Wl,-rpath," + libs, "-ltorch_python", "-ltorch_cuda", "-ltorch_cpu",
             "-lc10"], force)


def _sources():
    units = sorted(f for f in os.listdir(CSRC) if f.endswith(".cu"))
    deps = sorted(f for f in os.listdir(CSRC) if f.endswith((".cuh", ".h")))
    return units, deps


def _digest(units, deps, extra) -> str:
    h = hashlib.sha256()
    for name in units + deps:
        with open(os.path.join(CSRC, name), "rb") as f:
            h.update(name.encode() + b"\0" + f.read())
    with open(os.path.join(INCLUDE, "csr_spmm.h"), "rb") as f:
        h.update(f.read())
    h.update(" ".join(NVCC_FLAGS + LINK_FLAGS + list(extra)).encode())
    return h.hexdigest()


def build(verbose: bool = False, force: bool = False, extra_flags=(), out: str = LIB,
          flag_units=None) -> str:
    """Compile and link the library if anything changed; return its path.

    ``extra_flags`` (e.g. -D tuning macros) and ``out`` build a variant
    library elsewhere, with its own object directory.  With ``flag_units``
    (names of .cu files) only those units are compiled with ``extra_flags``;
    the others are linked from the library's own objects, which are brought
    up to date first."""
    units, deps = _sources()
    if flag_units is not None:
        flag_units = sorted(flag_units)
        missing = [u for u in flag_units if u not in units]
        if missing:
            raise ValueError(f"no such units: {missing}")
        if out == LIB:
            raise ValueError("a build restricted to some units needs its own output path")
        build(verbose=verbose)
    digest = _digest(units, deps, list(extra_flags) + ["units:"] + list(flag_units or []))
    stamp = out + ".sha256"
    obj_dir = OBJ_DIR if out == LIB else out + ".objs"
    if not force and os.path.exists(out) and os.path.exists(stamp):
        with open(stamp) as f:
            if f.read().strip() == digest:
                if out == LIB:
                    _lm_calls()
                    _torch_outputs()
                return out
    nvcc = _nvcc()
    os.makedirs(obj_dir, exist_ok=True)
    os.makedirs(os.path.dirname(out), exist_ok=True)

    def compile_one(unit):
        if flag_units is not None and unit not in flag_units:
            return os.path.join(OBJ_DIR, unit[:-3] + ".o")      # the library's own object
        obj = os.path.join(obj_dir, unit[:-3] + ".o")
        cmd = [nvcc] + NVCC_FLAGS + list(extra_flags) + ["-c", os.path.join(CSRC, unit), "-o", obj]
        if verbose:
            cmd += ["-Xptxas", "-v"]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {unit}:\n{r.stdout}\n{r.stderr}")
        if verbose and r.stderr:
            sys.stderr.write(r.stderr)
        return obj

    with ThreadPoolExecutor(max_workers=max(1, min(len(units), os.cpu_count() or 4))) as ex:
        modules = [ex.submit(m, force) for m in (_torch_outputs, _lm_calls) if out == LIB]
        objs = list(ex.map(compile_one, units))
    tmp = out + f".tmp{os.getpid()}"
    cmd = [nvcc] + ARCH + LINK_FLAGS + _runtime_path(nvcc) + ["-o", tmp] + objs
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, out)
    with open(stamp, "w") as f:
        f.write(digest + "\n")
    for m in modules:                        # a failure of theirs, now that the library is there
        m.result()
    return out


if __name__ == "__main__":
    print(build(verbose="-v" in sys.argv, force="-f" in sys.argv))
