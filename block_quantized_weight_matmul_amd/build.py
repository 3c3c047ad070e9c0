"""Build libqmm.so (the C-ABI library) for gfx950 with hipcc, and _calls.so (the binding's native calls) where it can be
built, in-tree.

    python block_quantized_weight_matmul_amd/build.py [-v]

Every HIP source under csrc/ is compiled to an object under _build/ (in
parallel), then linked into block_quantized_weight_matmul_amd/libqmm.so; csrc/calls.cpp,
host code against Python's and torch's headers, into _calls.so next to it.  The
library needs hipcc only.  Where _calls.so cannot be built (no torch, headers or
g++) it is left out, with a message, and the binding makes its calls through
ctypes.  Cross-compiles without a GPU.
"""

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
BUILD = os.path.join(ROOT, "_build")
LIB = os.path.join(PKG, "libqmm.so")
CALLS = os.path.join(PKG, "_calls.so")

ARCH = "gfx950"
FLAGS = [
    "-O3", "-std=c++17", f"--offload-arch={ARCH}", "-fPIC", "-Wall",
    # packed fp32 instructions are not generated for this library
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-I", INCLUDE, "-I", CSRC,
]


def hipcc():
    for cand in (os.environ.get("HIPCC"), shutil.which("hipcc"), "/opt/rocm/bin/hipcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("hipcc not found")


def sources():
    return sorted(os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith(".hip"))


def _compile(src, verbose):
    obj = os.path.join(BUILD, os.path.basename(src)[:-4] + ".o")
    cmd = [hipcc(), *FLAGS, "-c", src, "-o", obj]
    if verbose:
        print(" ".join(cmd), flush=True)
    r = subprocess.run(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True)
    out = "\n".join(ln for ln in r.stdout.splitlines() if "packed-fp32-ops" not in ln)
    if r.returncode != 0:
        raise RuntimeError(f"hipcc failed on {src}:\n{out}")
    if verbose and out.strip():
        print(out, flush=True)
    return obj


def _run(cmd, what, verbose):
    if verbose:
        print(" ".join(cmd), flush=True)
    r = subprocess.run(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"{what} failed:\n{r.stdout}")


def _compile_calls(verbose):
    import torch
    from torch.utils import cpp_extension
    obj = os.path.join(BUILD, "calls.host.o")
    paths = [INCLUDE, sysconfig.get_paths()["include"], *cpp_extension.include_paths()]
    built_for = f'-DQMM_BUILT_FOR="{torch.__version__} {sys.version_info[0]}.{sys.version_info[1]}"'
    _run(["g++", "-O2", "-std=c++17", "-fPIC", "-Wall", "-fvisibility=hidden", built_for, *(a for p in paths for a in ("-I", p)), "-c",
          os.path.join(CSRC, "calls.cpp"), "-o", obj], "g++ on calls.cpp", verbose)
    libs = [a for p in cpp_extension.library_paths() for a in ("-L", p)]
    return [obj, "-L", PKG, "-lqmm", *libs, "-ltorch_python", "-ltorch_cpu", "-lc10", "-Wl,-rpath,$ORIGIN"]


def _build_calls(compiled, verbose):
    """Link _calls.so of what `compiled` (a future of _compile_calls) has made.  One of an earlier build goes first: it may
    take another library's arguments."""
    if os.path.exists(CALLS):
        os.remove(CALLS)
    try:
        tmp = CALLS + ".tmp"
        _run(["g++", "-shared", "-o", tmp, *compiled.result()], "link of _calls.so", verbose)
        os.replace(tmp, CALLS)
    except (ImportError, OSError, RuntimeError) as e:
        print(f"_calls.so is not built; the attention calls go through ctypes: {e}", file=sys.stderr, flush=True)


def build(verbose=False, jobs=None):
    """Compile every source and link libqmm.so, and _calls.so where that can be built; returns the library's path."""
    os.makedirs(BUILD, exist_ok=True)
    srcs = sources()
    jobs = jobs or min(len(srcs), os.cpu_count() or 1, 16)
    with concurrent.futures.ThreadPoolExecutor(jobs) as ex:
        calls = ex.submit(_compile_calls, verbose)
        objs = list(ex.map(lambda s: _compile(s, verbose), srcs))
    tmp = LIB + ".tmp"
    _run([hipcc(), f"--offload-arch={ARCH}", "-shared", "-fPIC", *objs, "-o", tmp], "link", verbose)
    os.replace(tmp, LIB)
    _build_calls(calls, verbose)
    return LIB


if __name__ == "__main__":
    print(build(verbose="-v" in sys.argv))
