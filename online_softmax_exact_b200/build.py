"""Build libattn.so in-tree for sm_100a (nvcc cross-compiles; no GPU needed).

    python -m online_softmax_exact_b200.build [--verbose]
"""

from __future__ import annotations

import argparse
import os
import subprocess
import sys
from pathlib import Path

from ._abi import binding_target

PKG = Path(__file__).resolve().parent
CSRC = PKG / "csrc"
ROOT = PKG.parent
BUILD = ROOT / "_build"
LIB = PKG / "libattn.so"
BINDING = PKG / "_serving.so"  # the serving operators' torch binding, linked to libattn.so
BINDING_SOURCE = "serving_binding.cpp"
BINDING_STAMP = BUILD / "serving_binding.txt"  # what it was compiled against

ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
NVCC_FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "-Xcompiler", "-Wall",
              "--expt-relaxed-constexpr"]
SOURCES = ["attn_kernels.cu", "attn_api.cpp", "attn_noalloc.cu", "serve_kernels.cu", "serve_api.cpp"]
DEPS = ["sm100_ptx.cuh", "tma_host.h", "attn_fwd_kernel.cuh", "attn_merge_kernel.cuh",
        "attn_internal.h", "api_checks.h", "serve_params.h", "serve_ptx.cuh", "kv_plan_kernel.cuh",
        "qk_norm_rope_kernel.cuh", "kv4_layout.cuh", "kv4_copy_kernels.cuh", "kv4_fwd_kernel.cuh",
        "decode_common.cuh", "attn_window_kernel.cuh", "window_token_kernel.cuh"]


def nvcc() -> str:
    cand = os.environ.get("NVCC") or "/usr/local/cuda/bin/nvcc"
    return cand if os.path.exists(cand) else "nvcc"


def _stale(out: Path, sources) -> bool:
    if not out.exists():
        return True
    t = out.stat().st_mtime
    files = [CSRC / s for s in sources] + [ROOT / "include" / "attn.h"]
    return any(f.stat().st_mtime > t for f in files)


def build(force: bool = False, verbose: bool = False) -> Path:
    """Compile every CUDA source for sm_100a, link libattn.so next to this file, and the
    serving operators' torch binding beside it."""
    if force or _stale(LIB, SOURCES + DEPS):
        _build_lib(verbose)
    target = binding_target()
    built_for = BINDING_STAMP.read_text() if BINDING_STAMP.exists() else None
    if force or _stale(BINDING, [BINDING_SOURCE]) or built_for != target:
        _build_binding(target)
        BUILD.mkdir(exist_ok=True)
        BINDING_STAMP.write_text(target)
    return LIB


def _build_binding(target: str) -> None:
    import sysconfig

    import torch
    from torch.utils.cpp_extension import include_paths, library_paths

    cxx = os.environ.get("CXX") or "g++"
    libs = library_paths(device_type="cuda")
    tmp = BINDING.with_suffix(f".{os.getpid()}.tmp.so")
    cmd = [cxx, "-O2", "-std=c++17", "-fPIC", "-shared", "-Wall", "-Wno-unknown-pragmas",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           f'-DOSX_BUILT_FOR="{target}"',
           *[f"-isystem{p}" for p in include_paths(device_type="cuda")],
           f"-isystem{sysconfig.get_paths()['include']}", str(CSRC / BINDING_SOURCE), "-o", str(tmp),
           *[f"-L{p}" for p in libs], "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_cuda", "-ltorch",
           "-ltorch_python", f"-L{PKG}", "-l:libattn.so", "-Wl,-rpath,$ORIGIN"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"{cxx} failed on {BINDING_SOURCE}:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, BINDING)


def _build_lib(verbose: bool) -> None:
    BUILD.mkdir(exist_ok=True)
    objs = []
    for src in SOURCES:
        obj = BUILD / (Path(src).stem + ".o")
        cmd = [nvcc(), *ARCH, *NVCC_FLAGS, "-c", str(CSRC / src), "-o", str(obj)]
        if verbose and src.endswith(".cu"):
            cmd.insert(1, "-Xptxas=-v")
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {src}:\n{r.stdout}\n{r.stderr}")
        if verbose:
            sys.stderr.write(r.stdout + r.stderr)
        objs.append(str(obj))
    tmp = LIB.with_suffix(f".{os.getpid()}.tmp.so")
    cmd = [nvcc(), *ARCH, "-shared", "-o", str(tmp), *objs]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)


if __name__ == "__main__":
    ap = argparse.ArgumentParser()
    ap.add_argument("--verbose", action="store_true")
    ap.add_argument("--force", action="store_true")
    a = ap.parse_args()
    print(build(force=a.force or a.verbose, verbose=a.verbose))
