"""Build libfa.so in-tree with nvcc for sm_103a (one -gencode, sources compiled in
parallel, no cmake), and the compiled part of the Python binding with g++."""
from __future__ import annotations

import concurrent.futures as cf
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
BUILD_DIR = os.path.join(PKG, "_build")
LIB_PATH = os.path.join(PKG, "libfa.so")
BINDING_PATH = os.path.join(PKG, "_binding.so")
BINDING_KEY_PATH = os.path.join(BUILD_DIR, "_binding.key")
BINDING_SOURCE = os.path.join(CSRC, "binding.cpp")
SOURCES = ["fa_api.cu", "fa_fwd.cu", "fa_fwd_ring.cu", "fa_bwd.cu", "fa_bwd_q128.cu", "fa_bwd_pair.cu", "fa_merge.cu", "fa_noalloc.cu",
           "fa_varlen.cu", "fa_cache4.cu", "fa_cache4_attend.cu"]
HEADERS = ["fa_internal.h", "ptx.cuh", "exp2.cuh", "bwd_common.cuh", "fwd_common.cuh",
           "var_common.cuh", "cache4.cuh"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "-I", INCLUDE, "-I", CSRC]


def nvcc() -> str:
    for cand in (shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def _newer(path: str, deps: list[str]) -> bool:
    """Whether `path` is missing or one of `deps` is newer."""
    if not os.path.exists(path):
        return True
    t = os.path.getmtime(path)
    return any(os.path.getmtime(d) > t for d in deps)


def _run(cmd: list[str], what: str) -> str:
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"{what} failed:\n{r.stdout}\n{r.stderr}")
    return r.stderr


def _torch_dir() -> str:
    """torch's folder (found, not imported)."""
    return importlib.util.find_spec("torch").submodule_search_locations[0]


def _binding_key() -> str:
    """What _binding.so is linked to besides libfa.so: this Python and this torch's C++."""
    with open(os.path.join(_torch_dir(), "version.py"), encoding="utf-8") as f:
        return "\n".join((sysconfig.get_config_var("SOABI") or sys.version, _torch_dir(), f.read()))


def _binding_stale(header: str) -> bool:
    if _newer(BINDING_PATH, [BINDING_SOURCE, header]) or not os.path.exists(BINDING_KEY_PATH):
        return True
    with open(BINDING_KEY_PATH, encoding="utf-8") as f:
        return f.read() != _binding_key()


def _build_binding() -> None:
    """csrc/binding.cpp against this machine's torch and libfa.so."""
    torch = _torch_dir()
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(nvcc())))
    cxx = shutil.which("g++") or shutil.which("c++")
    if cxx is None:
        raise RuntimeError("g++ not found")
    inc = [INCLUDE, os.path.join(torch, "include"),
           os.path.join(torch, "include", "torch", "csrc", "api", "include"),
           os.path.join(cuda, "include"), sysconfig.get_paths()["include"]]
    tmp = BINDING_PATH + f".tmp{os.getpid()}"
    _run([cxx, "-O2", "-std=c++17", "-fPIC", "-shared", *[f"-I{d}" for d in inc], BINDING_SOURCE,
          "-o", tmp, f"-L{PKG}", "-l:libfa.so", "-Wl,-rpath,$ORIGIN",
          "-L" + os.path.join(torch, "lib"), "-ltorch_python", "-ltorch_cpu", "-lc10_cuda", "-lc10"],
         "g++ for binding.cpp")
    os.replace(tmp, BINDING_PATH)
    os.makedirs(BUILD_DIR, exist_ok=True)
    with open(BINDING_KEY_PATH + f".tmp{os.getpid()}", "w", encoding="utf-8") as f:
        f.write(_binding_key())
    os.replace(f.name, BINDING_KEY_PATH)


def build(force: bool = False, verbose: bool = False, extra: tuple[str, ...] = ()) -> str:
    header = os.path.join(INCLUDE, "fa.h")
    if force or _newer(LIB_PATH, [os.path.join(CSRC, f) for f in SOURCES + HEADERS] + [header]):
        _build_library(verbose, extra)
    if force or _binding_stale(header):
        _build_binding()
    return LIB_PATH


def _build_library(verbose: bool, extra: tuple[str, ...]) -> None:
    os.makedirs(BUILD_DIR, exist_ok=True)
    cc = nvcc()

    def compile_one(src):
        obj = os.path.join(BUILD_DIR, src.replace(".cu", ".o"))
        cmd = [cc, *ARCH, *FLAGS, *extra, "-c", os.path.join(CSRC, src), "-o", obj]
        if verbose:
            cmd.insert(1, "-Xptxas=-v")
        return obj, _run(cmd, f"nvcc for {src}")

    with cf.ThreadPoolExecutor(max_workers=len(SOURCES)) as ex:
        results = list(ex.map(compile_one, SOURCES))
    if verbose:
        for _, log in results:
            sys.stderr.write(log)
    tmp = LIB_PATH + f".tmp{os.getpid()}"
    _run([cc, *ARCH, "-shared", "-o", tmp, *[o for o, _ in results]], "link")
    os.replace(tmp, LIB_PATH)


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
