"""Build libnvfp4.so (the HIP kernels and the C ABI) in-tree for gfx950, and
the reference streaming kernels bench.py measures the HBM ceiling with
(bench_ref/libstream_ref.so, not part of the library); and _calls.so, the short
way from torch tensors to the library's calls (host code, by g++ with Python's and
torch's headers).

hipcc compiles every .hip source under csrc/ (several at a time) into one
shared library next to this file. Flags:
  --offload-arch=gfx950                 CDNA4 only, no other targets
  -O3 -ffp-contract=off                 no fused multiply-add contraction, so
                                        every product / quotient is rounded once
  (no -ffast-math)                      IEEE division, fp32 denormals kept
  -target-feature -packed-fp32-ops      keep the compiler from emitting packed
                                        fp32 VALU forms
"""
from __future__ import annotations

import glob
import os
import subprocess
import tempfile
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
ROOT = os.path.dirname(HERE)


BENCH_REF = os.path.join(HERE, "bench_ref")
FLAGS = ["--offload-arch=gfx950", "-O3", "-std=c++17", "-fPIC", "-shared", "-ffp-contract=off",
         "-Wall", "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops"]


def library_path() -> str:
    """The in-tree libnvfp4.so."""
    return os.path.join(HERE, "libnvfp4.so")


def stream_ref_path() -> str:
    """The reference streaming kernels bench.py measures the HBM ceiling with."""
    return os.path.join(BENCH_REF, "libstream_ref.so")


def _hipcc(sources, out, includes, verbose):
    hipcc = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
    tmp = out + ".tmp"

    def run(cmd):
        if verbose:
            print(" ".join(cmd), flush=True)
        subprocess.run(cmd, check=True)

    inc = [x for i in includes for x in ("-I", i)]
    with tempfile.TemporaryDirectory() as d:
        objs = [os.path.join(d, f"{i}.o") for i in range(len(sources))]
        jobs = [[hipcc, *(f for f in FLAGS if f != "-shared"), *inc, "-c", s, "-o", o]
                for s, o in zip(sources, objs)]
        with ThreadPoolExecutor(max(1, min(8, os.cpu_count() or 1))) as pool:
            list(pool.map(run, jobs))
        run([hipcc, "--offload-arch=gfx950", "-fPIC", "-shared", *objs, "-o", tmp])
    os.replace(tmp, out)
    return out


def calls_path() -> str:
    """The in-tree _calls.so."""
    return os.path.join(HERE, "_calls.so")


def build_calls(verbose: bool = False) -> str:
    """After build_library: it links against libnvfp4.so beside it."""
    import sysconfig

    import torch
    from torch.utils import cpp_extension

    out = calls_path()
    lib = os.path.join(os.path.dirname(torch.__file__), "lib")
    inc = [sysconfig.get_paths()["include"], os.path.join(ROOT, "include"), *cpp_extension.include_paths()]
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-Wall", *(x for i in inc for x in ("-isystem", i)),
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch.compiled_with_cxx11_abi())}", os.path.join(HERE, "binding", "calls.cpp"),
           "-o", out + ".tmp", "-L", lib, "-ltorch_python", "-ltorch_cpu", "-lc10", "-L", HERE, "-l:libnvfp4.so",
           "-Wl,-rpath,$ORIGIN"]
    if verbose:
        print(" ".join(cmd), flush=True)
    subprocess.run(cmd, check=True)
    os.replace(out + ".tmp", out)
    return out


def build_library(verbose: bool = False, out: str = None, csrc: str = CSRC) -> str:
    return _hipcc(sorted(glob.glob(os.path.join(csrc, "*.hip"))),
                  out or library_path(), [os.path.join(ROOT, "include"), csrc], verbose)


def build_stream_ref(verbose: bool = False) -> str:
    return _hipcc([os.path.join(BENCH_REF, "stream_ref.hip")], stream_ref_path(), [], verbose)


if __name__ == "__main__":
    print(build_library(verbose=True))
    print(build_calls(verbose=True))
    print(build_stream_ref(verbose=True))
