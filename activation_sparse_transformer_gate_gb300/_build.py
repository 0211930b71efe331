"""Build libtwell.so in-tree with nvcc for sm_103a (GB300).

Each translation unit compiles in parallel to an object under ``_build/``, then
nvcc links the shared library next to this file.  Rebuilds only when a source
or header is newer than the library.

Besides the product library, two variants of the same sources serve the tests
and the benchmark only (they are never loaded by the Python binding's
entry points):

* ``libtwell_hooks.so`` -- adds three hooks (``TWELL_TEST_HOOKS``):
  the tensor-core GEMM engine with a plain fp32 epilogue, and the random-row
  gather probe that the benchmark reads the gather kernels against; and a count
  of CTA pairs that end before their last commits have arrived.
* ``libtwell_timeout.so`` -- the same hooks of the kernels, and the pipeline waits of the tensor-core kernels
  limited to 1 ns, so that every wait that is not satisfied at once runs out
  on a sane input and the timeout path (status, drain, exit) can be tested
  without a fault.
"""
from __future__ import annotations

import concurrent.futures as cf
import importlib.util
import os
import shutil
import subprocess
import sys
import sysconfig
from typing import Optional

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
OBJDIR = os.path.join(PKG, "_build")

SOURCES = ["twell_abi.cu", "pack.cu", "simt_gemm.cu", "updown.cu", "tc_gemm.cu", "backward.cu",
           "rowell.cu", "static_split.cu", "lm_abi.cu", "embed.cu", "rmsnorm.cu", "distill.cu",
           "q8.cu"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]

# variant -> (library file, extra sources, extra nvcc flags)
VARIANTS = {
    "": ("libtwell.so", [], []),
    "hooks": ("libtwell_hooks.so", ["probe.cu"], ["-DTWELL_TEST_HOOKS"]),
    "timeout": ("libtwell_timeout.so", [], ["-DTWELL_WAIT_LIMIT_NS=1ull", "-DTWELL_TEST_HOOKS"]),
}
LIB = os.path.join(PKG, VARIANTS[""][0])
# Python's argument marshalling of the operators around the FFN (csrc/lm_bind.cpp), a CPython
# extension against torch's headers, beside libtwell.so and linked to it
BINDING = os.path.join(PKG, "_lm.so")
STAMP = os.path.join(OBJDIR, "lib", "lm_bind.for")  # the Python and torch that it was built for


def lib_path(variant: str = "") -> str:
    return os.path.join(PKG, VARIANTS[variant][0])


def nvcc_path() -> str:
    for c in (os.environ.get("NVCC"), "/usr/local/cuda/bin/nvcc", shutil.which("nvcc")):
        if c and os.path.exists(c):
            return c
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libtwell.so")


def _deps():
    files = [os.path.join(CSRC, f) for f in os.listdir(CSRC)]
    files += [os.path.join(INCLUDE, f) for f in os.listdir(INCLUDE)]
    files.append(os.path.abspath(__file__))
    return files


def _stale(lib: str) -> bool:
    if not os.path.exists(lib):
        return True
    t = os.path.getmtime(lib)
    return any(os.path.getmtime(f) > t for f in _deps())


def _jobs(variant: str):
    name, extra_src, flags = VARIANTS[variant]
    objdir = os.path.join(OBJDIR, variant or "lib")
    return [(src, os.path.join(objdir, os.path.splitext(src)[0] + ".o"), flags)
            for src in SOURCES + extra_src], objdir, os.path.join(PKG, name)


def _torch_dir() -> Optional[str]:
    """Where the torch is that a binding can be built against; None without one, or without a C++
    compiler (the C library needs only nvcc)."""
    spec = importlib.util.find_spec("torch")
    if spec is None or not spec.submodule_search_locations or not shutil.which("g++"):
        return None
    path = list(spec.submodule_search_locations)[0]
    return path if os.path.exists(os.path.join(path, "lib", "libc10_cuda.so")) else None


def _binding_tag(torch_dir: str) -> str:
    """What a binding is good for: this Python and this torch."""
    with open(os.path.join(torch_dir, "version.py"), encoding="utf-8") as f:
        version = f.read()
    return f"{sysconfig.get_config_var('SOABI')}\n{torch_dir}\n{version}"


def _binding_stale() -> bool:
    torch_dir = _torch_dir()
    if torch_dir is None:
        return False
    if _stale(BINDING) or not os.path.exists(STAMP):
        return True
    with open(STAMP, encoding="utf-8") as f:
        return f.read() != _binding_tag(torch_dir)


def _binding_flags(torch_dir: str, nvcc: str):
    dirs = [os.path.join(torch_dir, "include"),
            os.path.join(torch_dir, "include", "torch", "csrc", "api", "include"),
            os.path.join(os.path.dirname(os.path.dirname(nvcc)), "include"),
            sysconfig.get_paths()["include"]]
    return [a for d in dirs for a in ("-isystem", d)]


def build(force: bool = False, verbose: bool = False, extra_flags=(), variants=("",)) -> str:
    """Build the requested library variants ("" = libtwell.so); returns the
    path of the first one."""
    todo = [v for v in variants
            if force or _stale(lib_path(v)) or (v == "" and _binding_stale())]
    if not todo:
        return lib_path(variants[0])
    nvcc = nvcc_path()
    common = ARCH + ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-I", INCLUDE,
                     "-I", CSRC, "--expt-relaxed-constexpr"] + list(extra_flags)

    def compile_one(job):
        src, obj, flags = job
        if src.endswith(".cpp"):
            cmd = ["g++", "-c", os.path.join(CSRC, src), "-o", obj, "-O2", "-std=c++17", "-fPIC",
                   "-I", INCLUDE] + flags
        else:
            cmd = [nvcc, "-c", os.path.join(CSRC, src), "-o", obj] + common + flags
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"{cmd[0]} failed for {src}:\n{r.stdout}\n{r.stderr}")
        if verbose and (r.stdout or r.stderr):
            print(r.stdout + r.stderr, file=sys.stderr)
        return obj

    plans = []
    jobs = []
    for v in todo:
        js, objdir, lib = _jobs(v)
        os.makedirs(objdir, exist_ok=True)
        plans.append((js, lib))
        jobs += js
    torch_dir = _torch_dir() if "" in todo else None
    bind_obj = os.path.join(OBJDIR, "lib", "lm_bind.o")
    if torch_dir:
        jobs.insert(0, ("lm_bind.cpp", bind_obj, _binding_flags(torch_dir, nvcc)))
    workers = max(1, min(len(jobs), os.cpu_count() or 8))
    with cf.ThreadPoolExecutor(max_workers=workers) as ex:
        list(ex.map(compile_one, jobs))
    for js, lib in plans:
        tmp = lib + f".tmp{os.getpid()}"
        cmd = [nvcc, "-shared", "-o", tmp] + [o for _, o, _ in js] + ARCH + ["-ldl"]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc link failed:\n{r.stdout}\n{r.stderr}")
        os.replace(tmp, lib)
    if torch_dir:
        tmp = BINDING + f".tmp{os.getpid()}"
        libs = os.path.join(torch_dir, "lib")
        cmd = ["g++", "-shared", "-o", tmp, bind_obj, "-L", PKG, "-l:libtwell.so", "-L", libs,
               "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_python", "-Wl,-rpath,$ORIGIN"]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"g++ link failed:\n{r.stdout}\n{r.stderr}")
        os.replace(tmp, BINDING)
        with open(STAMP, "w", encoding="utf-8") as f:
            f.write(_binding_tag(torch_dir))
    elif "" in todo:
        print("no torch with CUDA, or no g++: the operators around the FFN have no Python binding",
              file=sys.stderr)
    return lib_path(variants[0])


def build_all(force: bool = False, verbose: bool = False) -> None:
    """The product library and both test variants, compiled together."""
    build(force=force, verbose=verbose, variants=tuple(VARIANTS))


if __name__ == "__main__":
    build_all(force="--force" in sys.argv, verbose=True)
    print("\n".join(lib_path(v) for v in VARIANTS))
