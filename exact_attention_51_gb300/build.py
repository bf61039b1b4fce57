"""Build the CUDA extension in place: exact_attention_51_gb300/libexact_attn_gb300.so.

Compiles every csrc/*.cu for sm_103a only (one -gencode), in parallel, and
links them into one shared library with the CUDA runtime linked statically, so
the library loads on hosts without a GPU (the runtime only looks for the driver
when a CUDA call is made).  No cmake, no torch extension machinery: the torch
binding of the per-token calls (csrc/python/binding.cpp -> _binding.so) is one
host file, compiled beside them and linked to the library.  The library does
not need it: it is linked first, and alone where there is no torch.
"""
from __future__ import annotations

import concurrent.futures as cf
import glob
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
LIB_NAME = "libexact_attn_gb300.so"
LIB_PATH = os.path.join(PKG, LIB_NAME)
BUILD_DIR = os.path.join(PKG, "_build")
BINDING_SRC = os.path.join(CSRC, "python", "binding.cpp")
BINDING_PATH = os.path.join(PKG, "_binding.so")
STAMP_PATH = os.path.join(BUILD_DIR, "binding.stamp")  # what _binding.so was compiled against

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC,-fvisibility=hidden", "--expt-relaxed-constexpr",
              "-I", INCLUDE, "-I", CSRC]


def nvcc() -> str:
    cand = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(cand):
        raise RuntimeError("nvcc not found")
    return cand


def _sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _headers():
    return sorted(glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(CSRC, "*.h"))
                  + glob.glob(os.path.join(INCLUDE, "*.h")))


def _compile(src: str, extra=()):
    obj = os.path.join(BUILD_DIR, os.path.basename(src) + ".o")
    cmd = [nvcc(), *ARCH, *NVCC_FLAGS, *extra, "-c", src, "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc failed for {src}:\n{r.stdout}\n{r.stderr}")
    return obj, r.stdout + r.stderr


def _compile_binding():
    """The torch binding's object file (host code; torch's headers)."""
    import torch
    obj = os.path.join(BUILD_DIR, "binding.cpp.o")
    inc = os.path.join(os.path.dirname(torch.__file__), "include")
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(nvcc())))
    cmd = [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-fvisibility=hidden",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           "-isystem", inc, "-isystem", os.path.join(inc, "torch", "csrc", "api", "include"),
           "-isystem", sysconfig.get_paths()["include"], "-isystem", os.path.join(cuda, "include"),
           "-I", INCLUDE, "-c", BINDING_SRC, "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"{cmd[0]} failed for {BINDING_SRC}:\n{r.stdout}\n{r.stderr}")
    return obj


def _link_binding(obj: str) -> None:
    import torch
    tmp = BINDING_PATH + f".tmp{os.getpid()}"
    cmd = [os.environ.get("CXX", "g++"), "-shared", "-o", tmp, obj,
           "-L", os.path.join(os.path.dirname(torch.__file__), "lib"),
           "-lc10", "-lc10_cuda", "-ltorch", "-ltorch_cpu", "-ltorch_cuda", "-ltorch_python",
           "-L", PKG, f"-l:{LIB_NAME}", "-Wl,-rpath,$ORIGIN"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, BINDING_PATH)


def _binding_stamp() -> str | None:
    """The torch (its version decides its C++ ABI) and the Python whose headers and internals the
    binding is compiled against; None where there is no torch, and so no binding."""
    spec = importlib.util.find_spec("torch")
    if spec is None:
        return None
    try:
        version = importlib.metadata.version("torch")
    except importlib.metadata.PackageNotFoundError:  # (run from a source tree)
        version = "of no package"
    return "\n".join([f"torch {version}", str(spec.origin),
                      str(sysconfig.get_config_var("SOABI"))])


def _read_stamp() -> str | None:
    try:
        with open(STAMP_PATH) as f:
            return f.read()
    except FileNotFoundError:
        return None


def up_to_date() -> bool:
    stamp = _binding_stamp()
    made = [LIB_PATH] + ([BINDING_PATH] if stamp else [])
    if not all(os.path.exists(f) for f in made):
        return False
    if stamp and _read_stamp() != stamp:
        return False
    t = min(os.path.getmtime(f) for f in made)
    return all(os.path.getmtime(f) <= t
               for f in _sources() + _headers() + [BINDING_SRC, __file__])


def build(force: bool = False, verbose_ptxas: bool = False, jobs: int | None = None) -> str:
    if not force and not verbose_ptxas and up_to_date():
        return LIB_PATH
    os.makedirs(BUILD_DIR, exist_ok=True)
    extra = ["-Xptxas", "-v"] if verbose_ptxas else []
    srcs = _sources()
    stamp = _binding_stamp()
    with cf.ThreadPoolExecutor(max_workers=jobs or min(len(srcs), os.cpu_count() or 4)) as ex:
        binding = ex.submit(_compile_binding) if stamp else None
        results = list(ex.map(lambda s: _compile(s, extra), srcs))
        if verbose_ptxas:
            for _, log in results:
                sys.stdout.write(log)
        tmp = LIB_PATH + f".tmp{os.getpid()}"
        cmd = [nvcc(), *ARCH, "-shared", "-cudart", "static", "-o", tmp,
               *[o for o, _ in results], "-lrt"]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
        os.replace(tmp, LIB_PATH)
        if binding is None:
            return LIB_PATH
        binding_obj = binding.result()
    if os.path.exists(STAMP_PATH):
        os.remove(STAMP_PATH)  # (of the binding that this one takes the place of)
    _link_binding(binding_obj)
    with open(STAMP_PATH, "w") as f:
        f.write(stamp)
    return LIB_PATH


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose_ptxas="-v" in sys.argv)
    print(LIB_PATH)
