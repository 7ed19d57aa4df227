"""Build libwf.so in-tree with nvcc for sm_100a, and _wf_torch.<versions>.so,
which checks torch tensors for the batch calls, with the host compiler.

    python -m chunk_causal_attention_block_b200.build [--verbose] [--no-torch]

A C program needs libwf.so alone: the other is left out with --no-torch, and
where there is no torch or no g++.  It reads the fields of torch's tensors
inline, so its name carries the torch and the Python that it was built for, and
one for others is neither loaded nor taken for up to date.  Objects go to
``_build/`` (git-ignored) and are rebuilt when a source or header is newer; the
shared libraries land next to this file so that they travel with the source
tree.
"""
from __future__ import annotations

import glob
import os
import shutil
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(ROOT, "_build")
LIB = os.path.join(PKG, "libwf.so")
TORCH_SRC = os.path.join(CSRC, "wf_torch.cc")

ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
NVCC_FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC,-O2", "--expt-relaxed-constexpr",
              "-I", INCLUDE, "-I", CSRC] + ARCH


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def _sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")) + glob.glob(os.path.join(CSRC, "*.cpp")))


def _headers():
    return glob.glob(os.path.join(CSRC, "*.h")) + glob.glob(os.path.join(CSRC, "*.cuh")) + \
        glob.glob(os.path.join(INCLUDE, "*.h"))


def torch_lib() -> str:
    """Path of the batch calls' tensor checks for the torch and the Python that run."""
    import torch
    version = torch.__version__.replace("+", "-")
    return os.path.join(PKG, f"_wf_torch.torch-{version}.{sysconfig.get_config_var('SOABI')}.so")


def build(verbose: bool = False, ptxas_verbose: bool = False, torch_calls: bool = True) -> str:
    os.makedirs(BUILD, exist_ok=True)
    hdr_mtime = max(os.path.getmtime(h) for h in _headers())
    objs = []
    for src in _sources():
        obj = os.path.join(BUILD, os.path.basename(src) + ".o")
        objs.append(obj)
        if os.path.exists(obj) and os.path.getmtime(obj) >= max(os.path.getmtime(src), hdr_mtime) \
                and not ptxas_verbose:
            continue
        cmd = [nvcc()] + NVCC_FLAGS + (["-Xptxas", "-v"] if ptxas_verbose else []) + ["-c", src, "-o", obj]
        if src.endswith(".cpp"):
            cmd = [nvcc()] + NVCC_FLAGS + ["-x", "cu", "-c", src, "-o", obj]
        if verbose:
            print(" ".join(cmd), flush=True)
        subprocess.run(cmd, check=True)
    if not os.path.exists(LIB) or os.path.getmtime(LIB) < max(os.path.getmtime(o) for o in objs):
        cmd = [nvcc()] + ARCH + ["-shared", "-o", LIB] + objs + ["-lcudart_static", "-lrt", "-ldl", "-lpthread"]
        if verbose:
            print(" ".join(cmd), flush=True)
        subprocess.run(cmd, check=True)
    if torch_calls:
        _build_torch_calls(verbose)
    return LIB


def _build_torch_calls(verbose: bool):
    try:
        import torch
    except ImportError:
        print("no torch: the batch calls' tensor checks are not built", file=sys.stderr)
        return
    if not shutil.which("g++"):
        print("no g++: the batch calls' tensor checks are not built", file=sys.stderr)
        return
    lib = torch_lib()
    newest = max(os.path.getmtime(f) for f in [TORCH_SRC, os.path.abspath(__file__)] + _headers())  # (flags: this file)
    if os.path.exists(lib) and os.path.getmtime(lib) >= newest:
        return
    # (the g++ on the path, whose C++ runtime torch shares; one that links the runtime statically cannot catch
    # torch's exceptions)
    root = os.path.dirname(torch.__file__)
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch.compiled_with_cxx11_abi())}", "-I", INCLUDE, "-I", CSRC,
           "-isystem", os.path.join(root, "include"),
           "-isystem", os.path.join(root, "include", "torch", "csrc", "api", "include"),
           "-isystem", sysconfig.get_paths()["include"], "-o", lib, TORCH_SRC,
           "-L", os.path.join(root, "lib"), "-ltorch_python", "-ltorch_cpu", "-lc10"]
    if verbose:
        print(" ".join(cmd), flush=True)
    subprocess.run(cmd, check=True)


if __name__ == "__main__":
    print(build(verbose="--verbose" in sys.argv, ptxas_verbose="--ptxas" in sys.argv,
                torch_calls="--no-torch" not in sys.argv))
