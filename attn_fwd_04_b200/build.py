"""Build libfa.so (the CUDA library behind include/fa.h) in-tree, for sm_100a, and
_calls.so (the binding's short way into it, host code only).

    python -m attn_fwd_04_b200.build [--force] [--verbose]

nvcc cross-compiles without a GPU.  The CUDA runtime is linked statically,
so the library loads on a machine without a driver (its calls then fail with
FA_ERR_CUDA); the driver's tensor-map encoder is looked up at run time.
"""
import os
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(PKG, "libfa.so")
CALLS = os.path.join(PKG, "_calls.so")
CALLS_TORCH = os.path.join(PKG, "_build", "calls.torch")  # what it was built against
SOURCES = ["api.cu", "fwd_sm100.cu", "bwd_sm100.cu", "decode_sm100.cu", "decode_noalloc.cu",
           "rope_sm100.cu", "append_sm100.cu", "decode_fp8_sm100.cu"]
HEADERS = ["fa_ptx.cuh", "fa_internal.h", "rope_row.cuh", "workspace.h"]

NVCC_FLAGS = [
    "-gencode", "arch=compute_100a,code=sm_100a",
    "-O3", "-std=c++17", "-lineinfo",
    "-Xcompiler", "-fPIC", "-Xcompiler", "-fvisibility=hidden",
    "--expt-relaxed-constexpr",
    "-cudart", "static",
]


def _nvcc() -> str:
    cand = os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "bin", "nvcc")
    return cand if os.path.exists(cand) else "nvcc"


def _stale(out: str, deps) -> bool:
    if not os.path.exists(out):
        return True
    t = os.path.getmtime(out)
    deps = [*deps, os.path.join(INCLUDE, "fa.h"), os.path.abspath(__file__)]
    return any(os.path.getmtime(p) > t for p in deps)


def _torch_of_calls() -> str:
    """The torch that CALLS was built against; empty: unknown."""
    try:
        with open(CALLS_TORCH) as f:
            return f.read().strip()
    except OSError:
        return ""


def _build_calls(force: bool, verbose: bool) -> None:
    """_calls.so, against the headers and libraries of the torch that runs this."""
    src = os.path.join(CSRC, "calls.cpp")
    import torch
    built_for = f"{torch.__version__} python {sys.version.split()[0]}"
    if not force and not _stale(CALLS, [src]) and _torch_of_calls() == built_for:
        return
    root = os.path.dirname(torch.__file__)
    headers = [os.path.join(root, "include"),
               os.path.join(root, "include", "torch", "csrc", "api", "include"),
               os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "include"),
               sysconfig.get_paths()["include"]]
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", "-I", INCLUDE]
    for h in headers:
        cmd += ["-isystem", h]
    cmd += [src, "-o", CALLS, "-L", os.path.join(root, "lib"), "-ltorch_python", "-ltorch",
            "-ltorch_cpu", "-lc10", "-lc10_cuda"]
    if verbose:
        print(" ".join(cmd), flush=True)
    subprocess.run(cmd, check=True)
    os.makedirs(os.path.dirname(CALLS_TORCH), exist_ok=True)
    with open(CALLS_TORCH, "w") as f:
        f.write(built_for + "\n")


def build(force: bool = False, verbose: bool = False) -> str:
    _build_calls(force, verbose)
    if not force and not _stale(LIB, [os.path.join(CSRC, f) for f in SOURCES + HEADERS]):
        return LIB
    objdir = os.path.join(PKG, "_build")
    os.makedirs(objdir, exist_ok=True)
    objs = []
    for src in SOURCES:
        obj = os.path.join(objdir, src.replace(".cu", ".o"))
        cmd = [_nvcc(), *NVCC_FLAGS, "-I", INCLUDE, "-I", CSRC, "-c",
               os.path.join(CSRC, src), "-o", obj]
        if verbose:
            cmd.insert(1, "-Xptxas=-v")
            print(" ".join(cmd), flush=True)
        subprocess.run(cmd, check=True)
        objs.append(obj)
    cmd = [_nvcc(), "-gencode", "arch=compute_100a,code=sm_100a", "-shared", "-cudart", "static",
           "-Xcompiler", "-fPIC", *objs, "-o", LIB]
    if verbose:
        print(" ".join(cmd), flush=True)
    subprocess.run(cmd, check=True)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="--verbose" in sys.argv))
