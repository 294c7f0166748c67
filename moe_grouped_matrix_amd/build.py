"""Build libgmm.so (the HIP kernels and the C ABI) for gfx950 with hipcc, and
_moe_ext.so (host code) beside it with the C++ compiler.

Run ``python -m moe_grouped_matrix_amd.build`` or call ``build()``; the
libraries are written next to this file.  libgmm.so needs hipcc alone;
_moe_ext.so needs a C++ compiler and torch's and Python's headers, and where it
cannot be built the binding does its work in Python."""
from __future__ import annotations

import os
import shutil
import subprocess
import sys
import warnings

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
LIB = os.path.join(HERE, "libgmm.so")
EXT = os.path.join(HERE, "_moe_ext.so")  # the Python side of gmm_moe.h and gmm_layer.h (host code over torch's C++ API)
SOURCES = [os.path.join(CSRC, n) for n in
           ("gmm_kernels.hip", "gmm_w8a8.hip", "gmm_stream.hip", "gmm_quant.hip", "gmm_moe.hip", "gmm_mxfp4.hip", "gmm_mxw.hip",
            "gmm_router.hip", "gmm_gmv.hip", "gmm_adamw.hip", "gmm_api.cpp", "gmm_moe_api.cpp", "gmm_layer_api.cpp")]

# Packed fp32 VALU instructions are kept out of the generated code.
HIPCC_FLAGS = ["--offload-arch=gfx950", "-O3", "-std=c++17", "-fPIC",
               "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
               "-Wno-unused-command-line-argument"]

# Per-source additions: the block-scaled fp8 kernel, the weight-streaming kernel
# and the products by expert id keep their MFMA results in ordinary VGPRs, where
# their scale folds read them.
EXTRA_FLAGS = {"gmm_w8a8.hip": ["-mllvm", "-amdgpu-mfma-vgpr-form"],
               "gmm_stream.hip": ["-mllvm", "-amdgpu-mfma-vgpr-form"],
               "gmm_gmv.hip": ["-mllvm", "-amdgpu-mfma-vgpr-form"]}


def hipcc() -> str:
    for cand in (os.environ.get("HIPCC"), "/opt/rocm/bin/hipcc", shutil.which("hipcc")):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("hipcc not found")


def _ext_command(out: str):
    """Compile and link csrc/moe_ext.cpp against the installed torch."""
    import sysconfig

    import torch
    from torch.utils import cpp_extension
    lib = os.path.join(os.path.dirname(torch.__file__), "lib")
    inc = [sysconfig.get_paths()["include"], os.path.join(HERE, "..", "include")] + cpp_extension.include_paths()
    return ([os.environ.get("CXX") or shutil.which("g++") or "c++", "-O2", "-std=c++17", "-fPIC", "-shared", "-w",
             "-D_GLIBCXX_USE_CXX11_ABI=%d" % int(torch.compiled_with_cxx11_abi())] + ["-I" + i for i in inc] +
            [os.path.join(CSRC, "moe_ext.cpp"), "-o", out, "-L" + lib, "-lc10", "-ltorch_cpu", "-ltorch_python"])


def _run(cmd, verbose):
    if verbose:
        print(" ".join(cmd), flush=True)
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError("hipcc failed:\n" + res.stdout + res.stderr)


def _build_ext(tag: str, verbose: bool):
    """Start compiling _moe_ext.so; returns a function that puts it in place,
    or takes an old one away and warns."""
    ext, proc, why = EXT + tag, None, ""
    try:
        cmd = _ext_command(ext)
        if verbose:
            print(" ".join(cmd), flush=True)
        proc = subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.PIPE, text=True)
    except (ImportError, OSError) as e:
        why = str(e)

    def finish(install: bool) -> None:
        out, err = proc.communicate() if proc else ("", why)
        if install and proc and proc.returncode == 0:
            os.replace(ext, EXT)
        elif install:
            # (one of another build may not fit this library)
            if os.path.exists(EXT):
                os.remove(EXT)
            warnings.warn("_moe_ext.so was not built; the token and fp4 operators are marshalled in Python:\n" + out + err)
        if os.path.exists(ext):
            os.remove(ext)
    return finish


def build(verbose: bool = False) -> str:
    """Compile every source to an object (in parallel), then link."""
    tag = ".tmp%d" % os.getpid()
    inc = "-I" + os.path.join(HERE, "..", "include")
    objs, procs = [], []
    for src in SOURCES:
        obj = os.path.join(CSRC, os.path.basename(src) + tag + ".o")
        cmd = [hipcc()] + HIPCC_FLAGS + EXTRA_FLAGS.get(os.path.basename(src), []) + [inc, "-c", src, "-o", obj]
        if verbose:
            print(" ".join(cmd), flush=True)
        procs.append((cmd, subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.PIPE, text=True)))
        objs.append(obj)
    finish_ext = _build_ext(tag, verbose)
    errors = []
    for cmd, pr in procs:
        out, err = pr.communicate()
        if pr.returncode != 0:
            errors.append(" ".join(cmd) + "\n" + out + err)
    built = False
    try:
        if errors:
            raise RuntimeError("hipcc failed:\n" + "\n".join(errors))
        tmp = LIB + tag
        _run([hipcc(), "--offload-arch=gfx950", "-shared", "-fPIC"] + objs + ["-o", tmp], verbose)
        os.replace(tmp, LIB)
        built = True
    finally:
        for o in objs:
            if os.path.exists(o):
                os.remove(o)
        finish_ext(built)
    return LIB


if __name__ == "__main__":
    print(build(verbose="-v" in sys.argv))
