"""Build libhlofusion.so in-tree for sm_103a (nvcc alone).

Every translation unit under csrc/ is compiled in parallel to an object file, then linked into
transpose_heroes_gb300/_lib/libhlofusion.so with the CUDA runtime linked statically. csrc/call.cc becomes
_lib/_hlocall.so, a CPython extension on top of it, compiled by the host compiler against the torch that is installed; without a
torch for CUDA it is left out, and the layer operators raise when they are called from Python.
"""

from __future__ import annotations

import concurrent.futures
import os
import shutil
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(PKG, "_build")
LIBDIR = os.path.join(PKG, "_lib")
LIB = os.path.join(LIBDIR, "libhlofusion.so")
CALL = os.path.join(LIBDIR, "_hlocall.so")

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-I", INCLUDE, "-I", CSRC]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libhlofusion")


def sources():
    return sorted(os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith(".cu"))


def headers():
    hs = [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith((".h", ".cuh", ".inc"))]
    return hs + [os.path.join(INCLUDE, f) for f in os.listdir(INCLUDE) if f.endswith(".h")]


def _stale(target: str, deps) -> bool:
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(d) > t for d in deps)


def build(verbose: bool = False, force: bool = False, ptxas_verbose: bool = False) -> str:
    os.makedirs(BUILD, exist_ok=True)
    os.makedirs(LIBDIR, exist_ok=True)
    srcs = sources()
    hdrs = headers()
    cc = nvcc()
    extra = ["-Xptxas", "-v"] if ptxas_verbose else []

    def compile_one(src):
        obj = os.path.join(BUILD, os.path.basename(src)[:-3] + ".o")
        if force or ptxas_verbose or _stale(obj, [src, *hdrs]):
            cmd = [cc, *ARCH, *NVCC_FLAGS, *extra, "-c", src, "-o", obj]
            r = subprocess.run(cmd, capture_output=True, text=True)
            if r.returncode != 0:
                raise RuntimeError(f"nvcc failed for {src}:\n{r.stdout}\n{r.stderr}")
            if verbose or ptxas_verbose:
                sys.stderr.write(r.stdout + r.stderr)
        return obj

    with concurrent.futures.ThreadPoolExecutor(max_workers=max(1, len(srcs) + 1)) as ex:
        call_obj = ex.submit(_compile_call, force)
        objs = list(ex.map(compile_one, srcs))
        call_obj = call_obj.result()
    if force or _stale(LIB, objs):
        tmp = LIB + f".tmp{os.getpid()}"
        cmd = [cc, *ARCH, "-shared", "-o", tmp, *objs, "-ldl"]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
        os.replace(tmp, LIB)
    if call_obj and (force or _stale(CALL, [call_obj]) or built_for() != call_abi()):
        _link_call(call_obj)
    return LIB


def call_abi() -> str:
    """What _hlocall.so is compiled for: the versions of torch and of Python's extensions. Empty without a torch for CUDA."""
    try:
        import torch
    except ImportError:
        return ""
    return f"torch {torch.__version__}, {sysconfig.get_config_var('SOABI')}" if torch.version.cuda else ""


def built_for(call: str | None = None) -> str:
    """call_abi() of when the extension was built."""
    path = (call or CALL) + ".abi"
    if not os.path.exists(path):
        return ""
    with open(path) as f:
        return f.read()


def _compile_call(force: bool) -> str | None:
    """The CPython extension that marshals the layer operators' calls (csrc/call.cc), against torch's headers; None without them."""
    src, obj = os.path.join(CSRC, "call.cc"), os.path.join(BUILD, "call.o")
    if not call_abi():
        return None
    if force or _stale(obj, [src, os.path.join(INCLUDE, "hlo_fusion.h")]) or built_for() != call_abi():
        import torch

        torch_include = os.path.join(os.path.dirname(torch.__file__), "include")
        cuda_include = os.path.join(os.path.dirname(os.path.dirname(nvcc())), "include")
        includes = [INCLUDE, sysconfig.get_paths()["include"], torch_include,
                    os.path.join(torch_include, "torch", "csrc", "api", "include"), cuda_include]
        abi = int(torch._C._GLIBCXX_USE_CXX11_ABI)
        cmd = [os.environ.get("CXX", "g++"), "-O2", "-std=c++20", "-fPIC", f"-D_GLIBCXX_USE_CXX11_ABI={abi}",
               *(f"-isystem{d}" if d != INCLUDE else f"-I{d}" for d in includes), "-c", src, "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"g++ failed for {src}:\n{r.stdout}\n{r.stderr}")
    return obj


def _link_call(obj: str) -> None:
    import torch

    torch_lib = os.path.join(os.path.dirname(torch.__file__), "lib")
    tmp = CALL + f".tmp{os.getpid()}"
    cmd = [os.environ.get("CXX", "g++"), "-shared", "-o", tmp, obj, "-L", LIBDIR, "-l:libhlofusion.so", "-Wl,-rpath,$ORIGIN",
           "-L", torch_lib, "-ltorch_python", "-ltorch_cpu", "-lc10", "-lc10_cuda", f"-Wl,-rpath,{torch_lib}"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, CALL)
    with open(CALL + ".abi", "w") as f:
        f.write(call_abi())


if __name__ == "__main__":
    print(build(verbose=True, ptxas_verbose="-v" in sys.argv, force="-f" in sys.argv))
