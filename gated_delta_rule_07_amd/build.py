"""Build libkda.so (HIP kernels + C ABI) for gfx950 with hipcc, in-tree.

Usage: ``python -m gated_delta_rule_07_amd.build`` (or ``build()`` from Python).
Each source compiles to an object in parallel, then one shared library is linked
next to this file, and beside it a small Python helper (_kda_args.so, host code), which the binding does
without where it cannot be built.  hipcc cross-compiles for gfx950 without a GPU present.
"""
from __future__ import annotations

import concurrent.futures as cf
import os
import shutil
import subprocess
import sys
import warnings
from pathlib import Path

PKG = Path(__file__).resolve().parent
CSRC = PKG / "csrc"
INCLUDE = PKG.parent / "include"
LIB = PKG / "libkda.so"
TEST_LIB = PKG / "libkda_testhooks.so"
ARGS_HELPER = PKG / "_kda_args.so"
OBJDIR = PKG / "_build"

SOURCES = ["kda_api.cpp", "kda_decode.hip", "kda_prefill.hip", "kda_prefill_pipe.hip", "kda_prep.hip",
           "kda_spec.hip", "kda_split.hip", "kda_cache_api.cpp", "kda_heads.hip", "kda_pages.hip", "kda_tree.hip"]

ARCH = "gfx950"
# Packed-fp32 VALU forms are disabled: plain fp32 code only.  Matrix-core
# accumulators stay in ordinary VGPRs: with one wave per SIMD the compiler would
# otherwise park them in AccVGPRs and copy them out for every VALU use.
DEVICE_FLAGS = ["-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops", "-mllvm", "-amdgpu-mfma-vgpr-form"]
COMMON = ["-O3", "-std=c++17", "-fPIC", f"--offload-arch={ARCH}", f"-I{INCLUDE}", f"-I{CSRC}"]


def hipcc() -> str:
    path = shutil.which("hipcc") or "/opt/rocm/bin/hipcc"
    if not os.path.exists(path):
        raise RuntimeError("hipcc not found; libkda needs ROCm to build")
    return path


def _compile(src: str, verbose: bool, defines=()) -> Path:
    out = OBJDIR / (Path(src).stem + ("_hooks" if defines else "") + ".o")
    cmd = [hipcc(), *COMMON, *DEVICE_FLAGS, *defines, "-c", str(CSRC / src), "-o", str(out)]
    if src.endswith(".cpp"):
        cmd[1:1] = ["-x", "hip"]
    if verbose:
        print(" ".join(cmd), flush=True)
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"hipcc failed for {src}:\n{r.stdout}\n{r.stderr}")
    return out


def _link(objs, lib: Path, verbose: bool) -> None:
    tmp = lib.with_suffix(".so.tmp%d" % os.getpid())
    cmd = [hipcc(), "-shared", "-fPIC", f"--offload-arch={ARCH}", *map(str, objs), "-o", str(tmp)]
    if verbose:
        print(" ".join(cmd), flush=True)
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, lib)


def _args_helper(verbose: bool) -> None:
    """The binding's argument helper: host code against the installed PyTorch's headers, whose version it carries."""
    import sysconfig

    import torch
    from torch.utils import cpp_extension as ext

    tmp = ARGS_HELPER.with_suffix(".so.tmp%d" % os.getpid())
    libs = ext.library_paths()
    cmd = [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-shared", str(CSRC / "kda_args.cpp"),
           *[f"-I{p}" for p in ext.include_paths()], f"-I{sysconfig.get_paths()['include']}",
           f'-DKDA_TORCH_VERSION="{torch.__version__}"',
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", *[f"-L{p}" for p in libs],
           "-ltorch_python", "-ltorch_cpu", "-lc10", f"-Wl,-rpath,{libs[0]}", "-o", str(tmp)]
    if verbose:
        print(" ".join(cmd), flush=True)
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"compiling kda_args.cpp failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, ARGS_HELPER)


def build(verbose: bool = False, jobs: int | None = None) -> Path:
    """Compile every source and link libkda.so; always rebuilds.

    Also links libkda_testhooks.so: the same kernels with the C ABI compiled
    with KDA_TEST_HOOKS, which adds kda_test_force_prefill (the tests use it to
    run the generic kernel on shapes the pipelined kernel would serve).  The
    product library carries no such switch.

    Where the argument helper cannot be built (no C++ compiler, no Python or
    PyTorch headers), an earlier build of it is removed and a warning says so:
    the binding then makes the same checks in Python."""
    OBJDIR.mkdir(exist_ok=True)
    jobs = jobs or min(len(SOURCES) + 1, max(1, os.cpu_count() or 1))
    units = [(s, ()) for s in SOURCES] + [("kda_api.cpp", ("-DKDA_TEST_HOOKS",))]
    with cf.ThreadPoolExecutor(max_workers=jobs) as ex:
        helper = ex.submit(_args_helper, verbose)
        objs = list(ex.map(lambda u: _compile(u[0], verbose, u[1]), units))
    _link(objs[:len(SOURCES)], LIB, verbose)
    _link([objs[-1]] + objs[1:len(SOURCES)], TEST_LIB, verbose)
    why = helper.exception()
    if why is not None:
        ARGS_HELPER.unlink(missing_ok=True)
        warnings.warn(f"the binding's argument helper was not built, its checks will run in Python: {why}", stacklevel=2)
    return LIB


if __name__ == "__main__":
    build(verbose="-v" in sys.argv)
    print(LIB)
