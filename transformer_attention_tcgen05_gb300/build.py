"""Builds libattn.so (the CUDA library behind include/libattn.h) and the native
part of the Python binding (_attn_native.so) in-tree.

    python -m transformer_attention_tcgen05_gb300.build [--force] [--verbose]

Each .cu under csrc/ compiles in parallel with nvcc for sm_103a only, then
links into transformer_attention_tcgen05_gb300/_build/libattn.so with the
CUDA runtime linked statically.  The binding (csrc/binding.cpp) compiles with
the host compiler against the installed torch and Python headers and links to
libattn.so beside it.  The library does not need the binding: where the binding
cannot be built, libattn.so is, and the entry points that go through the binding
raise.  Rebuilds only what changed, the binding also for another torch or Python.
"""
from __future__ import annotations

import concurrent.futures as cf
import glob
import os
import shutil
import subprocess
import sys
import sysconfig
import warnings

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
OUT = os.path.join(PKG, "_build")
LIB = os.path.join(OUT, "libattn.so")
BINDING = os.path.join(OUT, "_attn_native.so")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found (needed to build libattn for sm_103a)")


def _headers():
    return glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(CSRC, "*.h")) + \
        glob.glob(os.path.join(INCLUDE, "*.h"))


def _compile(src: str, obj: str, verbose: bool) -> str:
    cmd = [nvcc(), *ARCH, "-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC",
           "-Xcompiler", "-fvisibility=hidden", "--expt-relaxed-constexpr",
           "-I", INCLUDE, "-I", CSRC, "-c", src, "-o", obj]
    if verbose:
        cmd.insert(1, "-Xptxas=-v")
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc failed on {os.path.basename(src)}:\n{r.stderr}")
    return r.stderr


def _compile_binding(obj: str) -> str:
    import torch
    t = os.path.dirname(torch.__file__)
    cuda = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(nvcc()))), "include")
    abi = int(torch._C._GLIBCXX_USE_CXX11_ABI)
    cmd = [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-fvisibility=hidden",
           f"-D_GLIBCXX_USE_CXX11_ABI={abi}", "-I", INCLUDE, "-isystem", os.path.join(t, "include"),
           "-isystem", os.path.join(t, "include", "torch", "csrc", "api", "include"),
           "-isystem", sysconfig.get_paths()["include"], "-isystem", cuda,
           "-c", os.path.join(CSRC, "binding.cpp"), "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"{cmd[0]} failed on binding.cpp:\n{r.stderr}")
    return r.stderr


def _binding_for() -> str:
    """What a binding is built for: it fits no other torch or Python."""
    import torch
    return f"torch {torch.__version__} {torch._C._GLIBCXX_USE_CXX11_ABI} python {sysconfig.get_config_var('SOABI')}"


def _link_binding(obj: str) -> None:
    import torch
    lib = os.path.join(os.path.dirname(torch.__file__), "lib")
    tmp = BINDING + f".tmp{os.getpid()}"
    cmd = [os.environ.get("CXX", "g++"), "-shared", "-o", tmp, obj, "-L", OUT, "-lattn", "-L", lib,
           "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_python", "-Wl,-rpath,$ORIGIN"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link of the binding failed:\n{r.stderr}")
    os.replace(tmp, BINDING)


def build(force: bool = False, verbose: bool = False) -> str:
    """Compile (if stale) and link libattn.so and the binding; returns libattn.so's path.

    Raises if libattn.so cannot be built; a binding that cannot be is a warning."""
    os.makedirs(OUT, exist_ok=True)
    srcs = sorted(glob.glob(os.path.join(CSRC, "*.cu")))
    hdr_time = max([os.path.getmtime(h) for h in _headers()] + [0.0])
    jobs = []
    for s in srcs:
        o = os.path.join(OUT, os.path.basename(s)[:-3] + ".o")
        if force or verbose or not os.path.exists(o) or \
                os.path.getmtime(o) < max(os.path.getmtime(s), hdr_time):
            jobs.append((s, o))
    bsrc, bobj = os.path.join(CSRC, "binding.cpp"), os.path.join(OUT, "binding.o")
    stamp = bobj + ".for"                        # written once the binding is built
    made_for = open(stamp).read() if os.path.exists(stamp) else ""
    bind = force or not os.path.exists(bobj) or made_for != _binding_for() or \
        os.path.getmtime(bobj) < max(os.path.getmtime(bsrc), hdr_time)
    failed = None                                # why there is no binding
    if jobs or bind:
        with cf.ThreadPoolExecutor(max_workers=min(8, len(jobs) + 1)) as ex:
            bound = ex.submit(_compile_binding, bobj) if bind else None
            for (s, _), log in zip(jobs, ex.map(lambda j: _compile(j[0], j[1], verbose), jobs)):
                if verbose and log:
                    sys.stderr.write(f"== {os.path.basename(s)}\n{log}")
            if bound:
                failed = bound.exception()
    objs = [os.path.join(OUT, os.path.basename(s)[:-3] + ".o") for s in srcs]
    if jobs or not os.path.exists(LIB) or \
            os.path.getmtime(LIB) < max(os.path.getmtime(o) for o in objs):
        tmp = LIB + f".tmp{os.getpid()}"
        cmd = [nvcc(), *ARCH, "-shared", "-o", tmp, *objs, "-cudart", "static"]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"link failed:\n{r.stderr}")
        os.replace(tmp, LIB)
    if not failed and (bind or not os.path.exists(BINDING) or
                       os.path.getmtime(BINDING) < os.path.getmtime(bobj)):
        try:
            _link_binding(bobj)
            with open(stamp, "w") as f:
                f.write(_binding_for())
        except Exception as e:
            failed = e
    if failed:
        for old in (BINDING, bobj):              # what an earlier build left does not fit these sources
            if os.path.exists(old):
                os.remove(old)
        warnings.warn(f"the native binding was not built, its entry points will raise: {failed}",
                      RuntimeWarning, stacklevel=2)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="--verbose" in sys.argv))
