"""Compile libmaxsim.so (HIP kernels + C ABI) for gfx950 with hipcc, and the binding's Python extension
_fast.so with the host compiler, in-tree.

Usage: python -m late_interaction_retrieval_amd.build
"""
from concurrent.futures import ThreadPoolExecutor
import os
import subprocess
import sys
import sysconfig
import tempfile

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
LIB = os.path.join(HERE, "libmaxsim.so")
FAST = os.path.join(HERE, "_fast.so")
SOURCES = ["fwd.hip", "bwd.hip", "topk.hip", "ooc.hip", "chamfer.hip", "noalloc.hip", "capi.cpp",
           "rmsnorm.hip", "quant.hip", "gemm_fp8.hip", "adamw.hip", "capi_encoder.cpp",
           "rope.hip", "attn_fwd.hip", "attn_bwd.hip", "distill.hip", "capi_layers.cpp"]

HIPCC_FLAGS = [
    "--offload-arch=gfx950",
    "-O3",
    "-std=c++17",
    "-fPIC",
    # fp32 products and sums are separate IEEE operations unless fmaf is asked for
    "-ffp-contract=off",
    # no packed fp32 VALU ops
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-Wno-unused-command-line-argument",
]
# inputs are finite: max needs no NaN canonicalisation (infinities are kept)
FINITE_FLAGS = ["-fno-honor-nans"]
# these pass NaN and infinity through as their formulas give them, or refuse them
SOURCE_FLAGS = {s: [] for s in ("rmsnorm.hip", "quant.hip", "gemm_fp8.hip", "adamw.hip", "capi_encoder.cpp",
                                   "rope.hip", "attn_fwd.hip", "attn_bwd.hip", "distill.hip", "capi_layers.cpp")}


def hipcc():
    rocm = os.environ.get("ROCM_PATH", "/opt/rocm")
    return os.path.join(rocm, "bin", "hipcc")


def _run(cmd, verbose):
    if verbose:
        print(" ".join(cmd), flush=True)
    r = subprocess.run(cmd, capture_output=True, text=True)
    out = "\n".join(l for l in (r.stdout + r.stderr).splitlines()
                    if "packed-fp32-ops" not in l)
    if r.returncode != 0:
        raise RuntimeError("hipcc failed:\n" + out)
    if verbose and out.strip():
        print(out)


def _compile(sources, lib, verbose, extra):
    """Each source to an object (several at a time), then one link."""
    tmp = lib + ".tmp%d" % os.getpid()
    with tempfile.TemporaryDirectory(prefix="maxsim_build_") as objs:
        def one(s):
            obj = os.path.join(objs, s + ".o")
            _run([hipcc()] + HIPCC_FLAGS + SOURCE_FLAGS.get(s, FINITE_FLAGS) + list(extra) +
                 ["-I", os.path.join(ROOT, "include"), "-I", CSRC, "-c", os.path.join(CSRC, s), "-o", obj], verbose)
            return obj

        with ThreadPoolExecutor(max_workers=4) as pool:
            done = list(pool.map(one, sources))
        _run([hipcc(), "--offload-arch=gfx950", "-shared", "-fPIC"] + done + ["-o", tmp], verbose)
    os.replace(tmp, lib)
    return lib


def _compile_fast(verbose):
    """The extension: torch's C++ tensors, and libmaxsim.so beside it."""
    import torch

    base = os.path.dirname(torch.__file__)
    rocm = os.environ.get("ROCM_PATH", "/opt/rocm")
    tmp = FAST + ".tmp%d" % os.getpid()
    _run(["g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-D__HIP_PLATFORM_AMD__=1", "-DUSE_ROCM=1",
          "-D_GLIBCXX_USE_CXX11_ABI=%d" % int(torch._C._GLIBCXX_USE_CXX11_ABI), "-w",
          "-I", os.path.join(ROOT, "include"), "-I", os.path.join(base, "include"),
          "-I", os.path.join(base, "include", "torch", "csrc", "api", "include"),
          "-I", sysconfig.get_paths()["include"], "-I", os.path.join(rocm, "include"),
          os.path.join(CSRC, "fast_binding.cpp"), "-o", tmp, "-L", HERE, "-lmaxsim", "-Wl,-rpath,$ORIGIN",
          "-L", os.path.join(base, "lib"), "-ltorch_python", "-ltorch_cpu", "-lc10", "-lc10_hip"], verbose)
    os.replace(tmp, FAST)


def build(verbose=False, extra=()):
    """Build libmaxsim.so and _fast.so."""
    _compile(SOURCES, LIB, verbose, extra)
    _compile_fast(verbose)
    return LIB


if __name__ == "__main__":
    build(verbose=True, extra=sys.argv[1:])
    print(LIB)
