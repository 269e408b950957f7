"""Builds libgqa_attn.so in-tree with nvcc for sm_103a, and the native half of
the Python binding.

Each CUDA translation unit under csrc/ is compiled by its own nvcc process (in
parallel) and the objects are linked into ``libgqa_attn.so`` next to this
file; ``csrc/torch_call.cpp`` becomes the extension module ``_torch_call``
beside it, for the Python and the torch that are there (without torch the
library alone is built, which needs neither).  Nothing is installed anywhere
else.

    python -m gqa_attention_kv_decode_gb300.build [--force] [--verbose]
"""

from __future__ import annotations

import argparse
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
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libgqa_attn.so")
CALL = os.path.join(PKG, "_torch_call" + sysconfig.get_config_var("EXT_SUFFIX"))

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
CFLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC,-fvisibility=hidden",
          "--expt-relaxed-constexpr", "-I", INCLUDE, "-I", CSRC]


def _nvcc():
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA 13 toolkit is required to build libgqa_attn.so")


def _sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _torch():
    try:
        import torch
    except (ImportError, OSError):  # (none, or one whose own libraries are missing)
        return None
    return torch


def _host_compile(obj, torch):
    """The command that compiles csrc/torch_call.cpp (host code, torch headers)."""
    inc = os.path.join(os.path.dirname(torch.__file__), "include")
    cuda = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(_nvcc()))), "include")
    return ["g++", "-O2", "-std=c++17", "-fPIC", "-fvisibility=hidden", f'-DGQA_TORCH_VERSION="{torch.__version__}"',
            "-I", INCLUDE, "-isystem", inc, "-isystem", os.path.join(inc, "torch", "csrc", "api", "include"),
            "-isystem", sysconfig.get_paths()["include"], "-isystem", cuda, "-c",
            os.path.join(CSRC, "torch_call.cpp"), "-o", obj]


def _host_link(obj, out, torch):
    lib = os.path.join(os.path.dirname(torch.__file__), "lib")
    return ["g++", "-shared", "-o", out, obj, "-L", PKG, "-lgqa_attn", "-Wl,-rpath,$ORIGIN", "-L", lib, "-lc10",
            "-lc10_cuda", "-ltorch_cpu", "-ltorch_python"]


def _headers():
    return glob.glob(os.path.join(INCLUDE, "*.h")) + [os.path.abspath(__file__)]


def _newer(out, deps) -> bool:
    return os.path.exists(out) and all(os.path.getmtime(p) <= os.path.getmtime(out) for p in deps)


def _lib_up_to_date() -> bool:
    return _newer(LIB, _sources() + glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(CSRC, "*.h"))
                  + _headers())


def _call_stamp():
    return os.path.join(BUILD, "torch_call.torch")  # the torch that the module was built for


def _call_up_to_date(torch) -> bool:
    if not _newer(CALL, [os.path.join(CSRC, "torch_call.cpp")] + _headers()) or not os.path.exists(_call_stamp()):
        return False
    with open(_call_stamp()) as f:
        return f.read() == torch.__version__


def up_to_date() -> bool:
    torch = _torch()
    return _lib_up_to_date() and (torch is None or _call_up_to_date(torch))


def build(force: bool = False, verbose: bool = False, ptxas_info: bool = False) -> str:
    torch = _torch()
    do_lib = force or not _lib_up_to_date()
    do_call = torch is not None and (force or not _call_up_to_date(torch))
    if not do_lib and not do_call:
        return LIB
    nvcc = _nvcc()
    os.makedirs(BUILD, exist_ok=True)
    procs = []
    objs = []

    def start(name, cmd):
        if verbose:
            print(" ".join(cmd), flush=True)
        procs.append((name, subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True)))

    def link(cmd, tmp, out):
        if verbose:
            print(" ".join(cmd), flush=True)
        subprocess.run(cmd, check=True)
        os.replace(tmp, out)

    for src in _sources() if do_lib else ():
        obj = os.path.join(BUILD, os.path.basename(src)[:-3] + ".o")
        objs.append(obj)
        start(src, [nvcc, *ARCH, *CFLAGS, "-c", src, "-o", obj] + (["-Xptxas", "-v"] if ptxas_info else []))
    call_obj = os.path.join(BUILD, "torch_call.o")
    if do_call:
        start("torch_call.cpp", _host_compile(call_obj, torch))
    failed = []
    for src, p in procs:
        out, _ = p.communicate()
        if out and (verbose or ptxas_info or p.returncode != 0):
            print(out, file=sys.stderr)
        if p.returncode != 0:
            failed.append(os.path.basename(src))
    if failed != [] and failed != ["torch_call.cpp"]:
        raise RuntimeError("the compiler failed on: " + ", ".join(failed))
    if do_lib:
        link([nvcc, *ARCH, "-shared", "-o", LIB + ".tmp", *objs], LIB + ".tmp", LIB)
    if failed:
        raise RuntimeError("the compiler failed on: " + ", ".join(failed) + " (the C library is built)")
    if do_call:
        link(_host_link(call_obj, CALL + ".tmp", torch), CALL + ".tmp", CALL)
        with open(_call_stamp(), "w") as f:
            f.write(torch.__version__)
    elif torch is None:
        print("no torch: the C library is built, the Python binding's module is not", file=sys.stderr)
    return LIB


if __name__ == "__main__":
    ap = argparse.ArgumentParser()
    ap.add_argument("--force", action="store_true")
    ap.add_argument("--verbose", action="store_true")
    ap.add_argument("--ptxas-info", action="store_true")
    a = ap.parse_args()
    print(build(force=a.force, verbose=a.verbose, ptxas_info=a.ptxas_info))
