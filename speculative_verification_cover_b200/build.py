"""Build libdd.so in place with nvcc for sm_100a (B200), and beside it
libdd_checked.so, the same source with the device index checks compiled in
(DD_CHECK_BOUNDS; include/dd.h, dd_bounds_checked), and the binding's compiled
part (host code; args_path()).

    python -m speculative_verification_cover_b200.build [--force] [-v]
"""
from __future__ import annotations

import importlib.metadata
import os
import shutil
import subprocess
import sys
import sysconfig
import warnings

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
OUT = os.path.join(HERE, "libdd.so")
OUT_CHECKED = os.path.join(HERE, "libdd_checked.so")
HEADER = os.path.join(os.path.dirname(HERE), "include", "dd.h")
ARGS_SOURCE = os.path.join(CSRC, "dd_args.cpp")

NVCC_FLAGS = [
    "-gencode", "arch=compute_100a,code=sm_100a",
    "-O3", "-lineinfo", "-std=c++17",
    "-Xcompiler", "-fPIC", "-shared",
    "--expt-relaxed-constexpr",
]


def _nvcc():
    for cand in (shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def sources():
    return sorted(os.path.join(CSRC, f) for f in os.listdir(CSRC)
                  if f.endswith((".cu", ".cuh", ".h"))) + [HEADER]


def args_path() -> str:
    """The binding's compiled part. It reads Python's and torch's objects, so one that was built
    for another Python or torch has another name and is not found."""
    try:
        torch_version = importlib.metadata.version("torch")
    except importlib.metadata.PackageNotFoundError:
        torch_version = "none"
    return os.path.join(HERE, f"_args.{sysconfig.get_config_var('SOABI')}-torch{torch_version}.so")


def up_to_date(out: str = OUT) -> bool:
    if not os.path.exists(out):
        return False
    t = os.path.getmtime(out)
    # the binding's part calls the library by the header's signatures
    return all(os.path.getmtime(s) <= t for s in ([ARGS_SOURCE, HEADER] if out == args_path() else sources()))


def _args_command(out):
    """g++ for the binding's argument checks, which read torch's tensors."""
    import torch
    root = os.path.dirname(torch.__file__)
    return [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-shared",
            f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
            "-I" + sysconfig.get_paths()["include"], "-isystem", os.path.join(root, "include"),
            "-isystem", os.path.join(root, "include", "torch", "csrc", "api", "include"),
            "-o", out, ARGS_SOURCE, "-L" + os.path.join(root, "lib"), "-ltorch_python", "-ltorch_cpu", "-lc10"]


def _left_out(args, e):
    if os.path.exists(args):  # older than its sources: not to be called
        os.remove(args)
    warnings.warn(f"the binding's compiled part was not built, without it the cached-decoding calls raise ImportError: {e}")


def build(force: bool = False, verbose: bool = False) -> str:
    """Compile whichever of the two libraries and the binding's compiled part is missing or
    older than a source (all at once), and return the path of libdd.so. Without Python's or
    torch's headers the binding's part is left out with a warning: the libraries and the
    verification step's calls do without it, the cached-decoding calls say what is missing."""
    jobs = []
    for out, extra in ((OUT, []), (OUT_CHECKED, ["-DDD_CHECK_BOUNDS"])):
        if not force and up_to_date(out):
            continue
        tmp = out + ".tmp"
        cmd = [_nvcc(), *NVCC_FLAGS, *extra, "-o", tmp, os.path.join(CSRC, "libdd.cu")]
        if verbose:
            cmd.insert(1, "-Xptxas=-v")
            print(" ".join(cmd), flush=True)
        jobs.append((subprocess.Popen(cmd), tmp, out, cmd))
    args = args_path()
    if force or not up_to_date(args):
        try:
            cmd = _args_command(args + ".tmp")
            jobs.append((subprocess.Popen(cmd), args + ".tmp", args, cmd))
        except (ImportError, OSError) as e:  # no torch, no compiler
            _left_out(args, e)
    failed = None
    for proc, tmp, out, cmd in jobs:
        if proc.wait() != 0:
            e = subprocess.CalledProcessError(proc.returncode, cmd)
            if out == args:
                _left_out(args, e)
            else:
                failed = failed or e
        else:
            os.replace(tmp, out)
    if failed:
        raise failed
    return OUT


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
