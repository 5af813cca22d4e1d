"""Builds libgdn.so in-tree with nvcc for sm_103a (one -gencode, translation units compiled
in parallel, static CUDA runtime), and _binding.so, the native argument marshalling of the decoding
operators, with the host compiler against this installation of torch.  Run as ``python -m chunked_prefill_gb300.build``."""
from __future__ import annotations

import glob
import os
import platform
import shutil
import subprocess
import sys
import sysconfig
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
ROOT = os.path.dirname(HERE)
LIB = os.path.join(HERE, "libgdn.so")
BUILD = os.path.join(ROOT, "_build")
# checked variant (-DGDN_CHECK): every output store tests its index against the tensor's
# extent and records ERR_BOUNDS instead of writing out of range; for tests, not for timing
LIB_CHECK = os.path.join(HERE, "libgdn_check.so")
BUILD_CHECK = os.path.join(ROOT, "_build_check")
BINDING = os.path.join(HERE, "_binding.so")
BINDING_FOR = os.path.join(BUILD, "_binding.txt")  # what the built one is for
BINDING_SRC = os.path.join(CSRC, "binding.cpp")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]


def nvcc() -> str:
    cand = os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "bin", "nvcc")
    return cand if os.path.exists(cand) else (shutil.which("nvcc") or "nvcc")


def flags(extra=()):
    return ARCH + ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC",
                   "--expt-relaxed-constexpr", "-I", os.path.join(ROOT, "include"), *extra]


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _stale(lib) -> bool:
    if not os.path.exists(lib):
        return True
    t = os.path.getmtime(lib)
    deps = sources() + glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(CSRC, "*.h"))
    deps.append(os.path.join(ROOT, "include", "gdn.h"))
    return any(os.path.getmtime(d) > t for d in deps)


def _binding_made_for() -> str:
    """What _binding.so is compiled against: it can be loaded by no other torch or Python."""
    import torch
    return f"torch {torch.__version__} ({os.path.dirname(torch.__file__)}), {sys.implementation.cache_tag} {platform.machine()}\n"


def _binding_stale() -> bool:
    deps = [BINDING_SRC, os.path.join(ROOT, "include", "gdn.h")]
    if not os.path.exists(BINDING) or any(os.path.getmtime(d) > os.path.getmtime(BINDING) for d in deps):
        return True
    if not os.path.exists(BINDING_FOR):
        return True
    with open(BINDING_FOR) as f:
        return f.read() != _binding_made_for()


def build_binding(verbose: bool = False) -> str:
    import torch
    base = os.path.dirname(torch.__file__)
    cuda = os.path.dirname(os.path.dirname(nvcc()))
    tmp = BINDING + f".tmp{os.getpid()}"
    cmd = [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-shared",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           "-I", os.path.join(base, "include"), "-I", os.path.join(base, "include", "torch", "csrc", "api", "include"),
           "-I", sysconfig.get_paths()["include"], "-I", os.path.join(cuda, "include"), BINDING_SRC, "-o", tmp,
           "-L", os.path.join(base, "lib"), "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_cuda", "-ltorch_python"]
    if verbose:
        print(" ".join(cmd), flush=True)
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"{cmd[0]} failed for {BINDING_SRC}:\n{r.stderr}")
    os.replace(tmp, BINDING)
    os.makedirs(BUILD, exist_ok=True)
    with open(BINDING_FOR, "w") as f:
        f.write(_binding_made_for())
    return BINDING


def build(force: bool = False, verbose: bool = False, ptxas_v: bool = False,
          checked: bool = False) -> str:
    lib, bdir = (LIB_CHECK, BUILD_CHECK) if checked else (LIB, BUILD)
    os.makedirs(bdir, exist_ok=True)
    srcs = sources()
    objs = [os.path.join(bdir, os.path.basename(s) + ".o") for s in srcs]
    binding = (lambda: build_binding(verbose)) if force or _binding_stale() else (lambda: None)
    if not force and not _stale(lib):
        binding()
        return lib
    extra = (["-Xptxas", "-v"] if ptxas_v else []) + (["-DGDN_CHECK"] if checked else [])

    def compile_one(so):
        src, obj = so
        cmd = [nvcc(), *flags(extra), "-c", src, "-o", obj]
        if verbose:
            print(" ".join(cmd), flush=True)
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed for {src}:\n{r.stderr}")
        return r.stderr

    with ThreadPoolExecutor(max_workers=len(srcs) + 1) as ex:
        side = ex.submit(binding)
        logs = list(ex.map(compile_one, zip(srcs, objs)))
        side.result()
    if ptxas_v:
        for s, log in zip(srcs, logs):
            print(f"== {os.path.basename(s)}\n{log}")
    tmp = lib + f".tmp{os.getpid()}"
    cmd = [nvcc(), *ARCH, "-shared", "-o", tmp, *objs]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stderr}")
    os.replace(tmp, lib)
    return lib


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True, ptxas_v="-v" in sys.argv,
                checked="--checked" in sys.argv))
