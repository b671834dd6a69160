"""Builds libattn.so (the CUDA library behind include/attn.h) in-tree with nvcc
for sm_103a.  Translation units compile in parallel; the link uses the static
CUDA runtime, so the library loads on machines without a GPU driver (its
entry points then report ATTN_ERR_CUDA on the first CUDA call).  Beside it,
with g++ and torch's headers, the extension module that marshals the 4-bit
cache's and the rotary positions' calls (csrc/calls.cpp).  Nothing depends on
that module but the time those calls take: where it cannot be built, the build
says so and the library is there all the same."""
from __future__ import annotations

import glob
import os
import shutil
import subprocess
import sys
import sysconfig
import warnings

import torch

PKG = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(os.path.dirname(PKG), "include")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libattn.so")
CALLS = os.path.join(PKG, f"_calls-{torch.__version__}.so")  # by torch's version: it uses torch's C++ interface

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", f"-I{INCLUDE}"]
# Per-file flags.  dsa_select.cu computes scores whose exact fp32 rounding
# decides an index set: no multiply may be fused into an add there, including
# the packed f32x2 pairs (which an explicit .rn does not keep apart).
FILE_FLAGS = {"dsa_select.cu": ["-fmad=false"]}


def _nvcc() -> str:
    for cand in (shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libattn.so")


def sources() -> list[str]:
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _newer(made: str, inputs: list[str]) -> bool:
    """Whether `made` is there and no older than its inputs."""
    return os.path.exists(made) and all(os.path.getmtime(f) <= os.path.getmtime(made) for f in inputs)


def _library_up_to_date() -> bool:
    return _newer(LIB, sources() + glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(CSRC, "*.h")) +
                  glob.glob(os.path.join(INCLUDE, "*.h")) + [os.path.abspath(__file__)])


def _calls_up_to_date() -> bool:
    return _newer(CALLS, [os.path.join(CSRC, "calls.cpp"), *glob.glob(os.path.join(INCLUDE, "*.h")), os.path.abspath(__file__)])


def up_to_date() -> bool:
    return _library_up_to_date() and _calls_up_to_date()


def _start_calls(out: str):
    """g++ on csrc/calls.cpp, as a running process that writes the extension module to `out`."""
    base = os.path.dirname(torch.__file__)
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(_nvcc())))
    include = [sysconfig.get_paths()["include"], os.path.join(base, "include"),
               os.path.join(base, "include", "torch", "csrc", "api", "include"), os.path.join(cuda, "include")]
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-shared", f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           *(f"-I{i}" for i in include), os.path.join(CSRC, "calls.cpp"), "-o", out, f"-L{os.path.join(base, 'lib')}",
           "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_python"]
    return subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True)


def build(force: bool = False, verbose: bool = False, extra_flags: tuple[str, ...] = (),
          out_path: str | None = None) -> str:
    """Compile every csrc/*.cu for sm_103a and link libattn.so; returns its path.
    ``extra_flags`` / ``out_path`` build a variant next to (not over) the
    default library, e.g. with a different -D setting."""
    lib = out_path or LIB
    calls = None  # the running compiler of the extension module
    if out_path is None and (force or not _calls_up_to_date()):
        made = CALLS + f".tmp{os.getpid()}"
        try:
            calls = _start_calls(made)
        except (OSError, RuntimeError) as e:  # no g++, no toolkit
            _without_calls(str(e))
    try:
        if force or extra_flags or out_path is not None or not _library_up_to_date():
            _build_library(lib, extra_flags, out_path, verbose)
    finally:
        if calls is not None:
            out, _ = calls.communicate()
            if calls.returncode != 0:
                _without_calls(out)
            else:
                if out and verbose:
                    sys.stdout.write(out)
                os.replace(made, CALLS)
    return lib


def _without_calls(why: str):
    """Says that there is no extension module; one of other sources does not stay."""
    if os.path.exists(CALLS):
        os.remove(CALLS)
    warnings.warn(f"{CALLS} was not built: the calls it would marshal go through Python, 5 to 10 us longer each\n{why}",
                  RuntimeWarning, stacklevel=3)


def _build_library(lib: str, extra_flags: tuple[str, ...], out_path: str | None, verbose: bool):
    nvcc = _nvcc()
    objdir = BUILD if out_path is None else os.path.join(BUILD, "variant_" + os.path.basename(lib))
    os.makedirs(objdir, exist_ok=True)
    procs = []
    for src in sources():
        obj = os.path.join(objdir, os.path.basename(src) + ".o")
        cmd = [nvcc, *ARCH, *NVCC_FLAGS, *FILE_FLAGS.get(os.path.basename(src), []), *extra_flags, "-c", src,
               "-o", obj]
        if verbose:
            print(" ".join(cmd), flush=True)
        procs.append((src, obj, subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT,
                                                 text=True)))
    objs, failed = [], []
    for src, obj, pr in procs:
        out, _ = pr.communicate()
        if out and (verbose or pr.returncode):
            sys.stdout.write(out)
        if pr.returncode != 0:
            failed.append(src)
        objs.append(obj)
    if failed:
        raise RuntimeError(f"nvcc failed for {failed}")
    tmp = lib + f".tmp{os.getpid()}"
    subprocess.run([nvcc, "-shared", *ARCH, "-o", tmp, *objs], check=True)
    os.replace(tmp, lib)


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True))
