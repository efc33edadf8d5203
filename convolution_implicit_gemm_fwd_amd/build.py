"""Build libconvimg.so (HIP, gfx950) and _rows.so in-tree.

``python -m convolution_implicit_gemm_fwd_amd.build`` compiles the HIP
translation units with hipcc for gfx950 only (each with its own extra flags)
and links them into one shared library next to this file; and, where torch is
installed, the host-only module that calls it from torch (csrc/rows_ext.cpp)
with the C++ compiler.  The library needs neither torch nor the module.
"""
from __future__ import annotations

import os
import shutil
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(PKG, "libconvimg.so")
EXT = os.path.join(PKG, "_rows.so")
# (source, extra hipcc flags): the weight-backward kernel keeps its MFMA
# accumulators in VGPRs (fewer register copies in its loop, measured)
UNITS = [(os.path.join(CSRC, "conv2d_fwd.hip"), []),
         (os.path.join(CSRC, "conv2d_wgrad.hip"), ["-mllvm", "-amdgpu-mfma-vgpr-form"]),
         (os.path.join(CSRC, "layer_norm.hip"), []),
         (os.path.join(CSRC, "mxfp4.hip"), [])]
SOURCES = [u[0] for u in UNITS]
DEPENDS = SOURCES + [os.path.join(CSRC, h) for h in ("igemm_common.hpp", "igemm_regs.hpp", "igemm_pipe.hpp", "igemm_patch.hpp", "igemm_strip.hpp", "igemm_window.hpp", "igemm_resident.hpp", "igemm_image.hpp", "igemm_dgrad.hpp", "igemm_wgrad.hpp", "igemm_layout.hpp", "row_common.hpp", "mxfp4_quant.hpp", "mxfp4_gemm.hpp", "mxfp4_few.hpp", "rows_ext.cpp")] + [os.path.join(INCLUDE, "convimg.h")]

ARCH = "gfx950"
HIPCC_FLAGS = [
    "--offload-arch=" + ARCH,
    "-O3",
    "-std=c++17",
    "-fPIC",
    "-shared",
    "-Wall",
    # packed fp32 instructions stay off in every kernel
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
]


def hipcc() -> str:
    for c in (os.environ.get("HIPCC"), "/opt/rocm/bin/hipcc", shutil.which("hipcc")):
        if c and os.path.exists(c):
            return c
    raise RuntimeError("hipcc not found; the HIP library cannot be built")


def ext_command(out: str):
    """The command that compiles the torch module (host code only), None
    without torch."""
    import importlib.util
    import sysconfig

    spec = importlib.util.find_spec("torch")
    if spec is None:
        return None
    torch = spec.submodule_search_locations[0]
    cxx = os.environ.get("CXX") or shutil.which("g++") or "/opt/rocm/llvm/bin/clang++"
    return [cxx, "-O2", "-std=c++17", "-fPIC", "-shared", "-Wall", "-D__HIP_PLATFORM_AMD__=1", "-DUSE_ROCM",
            "-isystem", os.path.join(torch, "include"),
            "-isystem", os.path.join(torch, "include", "torch", "csrc", "api", "include"),
            "-isystem", "/opt/rocm/include", "-isystem", sysconfig.get_paths()["include"], "-I", INCLUDE,
            os.path.join(CSRC, "rows_ext.cpp"), "-o", out, "-L" + os.path.join(torch, "lib"),
            "-ltorch_python", "-ltorch_hip", "-ltorch_cpu", "-lc10", "-lc10_hip"]


def build(verbose: bool = False, extra_flags=()) -> str:
    """Compile the library (always) and return its path.  A failure of the
    torch module is raised after the library is in place."""
    tag = "%d" % os.getpid()
    # the host pass does not know the packed-fp32 feature and says so
    noise = "'-packed-fp32-ops' is not a recognized feature"
    tmp, ext_tmp = LIB + ".tmp" + tag, EXT + ".tmp" + tag
    objs = [os.path.join(PKG, os.path.basename(src) + ".%s.o" % tag) for src, _ in UNITS]
    flags_c = [f for f in HIPCC_FLAGS if f != "-shared"]
    units = [[hipcc(), *flags_c, *flags, *extra_flags, "-I", INCLUDE, "-c", src, "-o", obj]
             for (src, flags), obj in zip(UNITS, objs)]
    link = [hipcc(), "--offload-arch=" + ARCH, "-shared", "-fPIC", *objs, "-o", tmp]
    ext = ext_command(ext_tmp)

    def start(cmd):
        if verbose:
            print(" ".join(cmd), flush=True)
        return subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True)

    def finish(p):
        """What the compiler says if it fails, else None."""
        out, _ = p.communicate()
        msgs = "\n".join(ln for ln in out.splitlines() if noise not in ln)
        if p.returncode != 0:
            return msgs
        if verbose and msgs:
            print(msgs)
        return None

    try:
        # the translation units compile in parallel
        procs = [start(cmd) for cmd in units]
        ext_proc = ext_failed = None
        if ext is not None:
            try:
                ext_proc = start(ext)
            except OSError as e:
                ext_failed = str(e)
        failed = [m for m in map(finish, procs) if m is not None]
        if ext_proc is not None:
            ext_failed = finish(ext_proc)
        if not failed:
            m = finish(start(link))
            failed = [] if m is None else [m]
        if failed:
            raise RuntimeError("hipcc failed:\n" + "\n".join(failed))
        os.replace(tmp, LIB)
        if ext_failed is not None:
            raise RuntimeError("libconvimg.so is built; the compiler of _rows.so failed:\n" + ext_failed)
        if ext is not None:
            os.replace(ext_tmp, EXT)
    finally:
        for o in (*objs, tmp, ext_tmp):
            if os.path.exists(o):
                os.remove(o)
    return LIB


if __name__ == "__main__":
    print(build(verbose=True, extra_flags=sys.argv[1:]))
