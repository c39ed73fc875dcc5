"""Build the gfx950 MoE layer library (libmoe_wq.so) and the one that it is linked
to (libmoe_wq_i8.so, 8-bit products) in-tree with hipcc."""
from __future__ import annotations

import concurrent.futures
import os
import subprocess
import tempfile

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
ROOT = os.path.dirname(HERE)
LIB = os.path.join(HERE, "libmoe_wq.so")
LIB_I8 = os.path.join(HERE, "libmoe_wq_i8.so")
HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
SOURCES = ["abi.cpp", "route.hip", "permute.hip", "quant.hip", "ffn.hip",
           "ffn_decode.hip", "ffn_bitplane.hip", "ffn_prefill.hip",
           "combine.hip", "alloc.hip", "cache.hip", "cache.cpp", "noalloc.hip", "retile.hip",
           "norm.hip", "block_out.hip", "sort.hip", "linear.hip", "quant_i8.hip", "gated_ffn.hip"]
SOURCES_I8 = ["linear_i8.hip"]
# Packed fp32 VALU instructions stay disabled in every HIP build here.
# MFMA accumulators are allocated in ordinary VGPRs (not AGPRs): the kernels
# rescale and convert accumulators with VALU instructions, which would
# otherwise need a move to and from the AGPR file for every element.
FLAGS = ["--offload-arch=gfx950", "-O3", "-std=c++17", "-fPIC",
         "-Wall", "-Wno-unused-result", "-Xclang", "-target-feature",
         "-Xclang", "-packed-fp32-ops", "-mllvm", "-amdgpu-mfma-vgpr-form=1",
         "-I", os.path.join(ROOT, "include")]


def _run(what, cmd):
    r = subprocess.run(cmd, cwd=CSRC, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"{what} failed:\n" + r.stdout + r.stderr)
    return r.stderr


def _link(lib, objects, *more):
    _run(f"{os.path.basename(lib)} link",
         [HIPCC, "--offload-arch=gfx950", "-shared", "-fPIC", "-o", lib, *objects, *more])


def build(verbose: bool = False) -> str:
    sources = SOURCES + SOURCES_I8
    # beside the libraries, which are both replaced when both are there
    with tempfile.TemporaryDirectory(dir=os.path.dirname(LIB), prefix=".build_") as made:
        out = [os.path.join(made, s + ".o") for s in sources]

        def compile_one(s, o):
            return _run(f"{s} build", [HIPCC, *FLAGS, "-c", os.path.join(CSRC, s), "-o", o])

        jobs = int(os.environ.get("MAX_JOBS", 0)) or min(8, os.cpu_count() or 1)
        with concurrent.futures.ThreadPoolExecutor(jobs) as pool:
            for said in pool.map(compile_one, sources, out):
                if verbose:
                    print(said)
        n = len(SOURCES)
        lib, lib_i8 = (os.path.join(made, os.path.basename(p)) for p in (LIB, LIB_I8))
        _link(lib_i8, out[n:], "-Wl,-soname," + os.path.basename(LIB_I8))
        # found beside the library, here and wherever both are copied
        _link(lib, [*out[:n], lib_i8], "-Wl,-rpath,$ORIGIN")
        os.replace(lib_i8, LIB_I8)
        os.replace(lib, LIB)
    return LIB


if __name__ == "__main__":
    print(build(verbose=True))
