"""Build libsgmv.so, the HIP library behind the SGMV C ABI, for gfx950.

    python -m segmented_gather_gemv_sgmv_amd.build

compiles the sources of the C ABI (``csrc/*.hip``, which include the kernel
headers) side by side with hipcc and links them into ``libsgmv.so`` next to
this file.  Cross-compiles without a GPU.
"""
from __future__ import annotations

import os
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIBRARY = os.path.join(PKG, "libsgmv.so")
SOURCES = [os.path.join(CSRC, f) for f in ("sgmv_api.hip", "q4_api.hip", "q4_f32.hip", "q4_f16.hip",
                                           "q4_bf16.hip", "ffn_api.hip", "rope_api.hip")]
OBJECTS = os.path.join(PKG, "_build")
ARCH = "gfx950"

HIPCC_FLAGS = [
    f"--offload-arch={ARCH}",
    "-O3",
    "-std=c++17",
    "-fPIC",
    "-shared",
    # Keep the compiler from forming packed fp32 instructions (v_pk_*_f32).
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-Wall",
    "-Wno-unused-function",
]


def hipcc() -> str:
    rocm = os.environ.get("ROCM_PATH", "/opt/rocm")
    path = os.path.join(rocm, "bin", "hipcc")
    return path if os.path.exists(path) else "hipcc"


def _object(source: str, tag: str) -> str:
    return os.path.join(OBJECTS, os.path.basename(source)[:-len(".hip")] + tag + ".o")


def _compile_and_link(jobs, verbose: bool):
    """jobs: (flags, output, tag).  Every source of every job is compiled at
    the same time, then each job's objects are linked."""
    os.makedirs(OBJECTS, exist_ok=True)
    procs = []
    for flags, output, tag in jobs:
        for src in SOURCES:
            cmd = [hipcc(), *[f for f in flags if f != "-shared"], "-I", INCLUDE, "-I", CSRC, "-c",
                   "-o", _object(src, tag), src]
            if verbose:
                print(" ".join(cmd), flush=True)
            procs.append(subprocess.Popen(cmd))
    codes = [p.wait() for p in procs]
    if any(codes):
        raise subprocess.CalledProcessError(max(codes, key=abs), "hipcc")
    for flags, output, tag in jobs:
        cmd = [hipcc(), *flags, "-o", output + ".tmp", *[_object(src, tag) for src in SOURCES]]
        if verbose:
            print(" ".join(cmd), flush=True)
        subprocess.run(cmd, check=True)
        os.replace(output + ".tmp", output)


def build(output: str = LIBRARY, extra_flags=(), verbose: bool = False) -> str:
    _compile_and_link([([*HIPCC_FLAGS, *extra_flags], output, "")], verbose)
    return output


# The same library with its HOST code under AddressSanitizer, for the CPU
# tests of the C ABI's argument checks (no kernel runs there, so the device
# code is compiled unoptimised, which keeps the build short).  Loaded with
# the sanitizer runtime preloaded (ASAN_RUNTIME) and SGMV_LIBRARY pointing
# at it; never used on a GPU.
ASAN_LIBRARY = os.path.join(PKG, "libsgmv_asan.so")
ASAN_FLAGS = [
    f"--offload-arch={ARCH}",
    "-std=c++17",
    "-fPIC",
    "-shared",
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-Xarch_host", "-O1",
    "-Xarch_host", "-g",
    "-Xarch_host", "-fno-omit-frame-pointer",
    "-Xarch_host", "-fsanitize=address",
    "-Xarch_host", "-shared-libasan",
    "-Xarch_device", "-O0",
    "-w",
]


def asan_runtime() -> str:
    """Path of clang's shared AddressSanitizer runtime in the ROCm toolchain."""
    import glob
    rocm = os.environ.get("ROCM_PATH", "/opt/rocm")
    hits = sorted(glob.glob(os.path.join(rocm, "lib", "llvm", "lib", "clang", "*", "lib", "linux",
                                         "libclang_rt.asan-x86_64.so")))
    if not hits:
        raise FileNotFoundError("libclang_rt.asan-x86_64.so not found under " + rocm)
    return hits[-1]


def sources_mtime() -> float:
    paths = [os.path.join(CSRC, f) for f in os.listdir(CSRC)]
    paths += [os.path.join(INCLUDE, f) for f in os.listdir(INCLUDE)]
    return max(os.path.getmtime(p) for p in paths)


def build_asan(output: str = ASAN_LIBRARY, verbose: bool = False) -> str:
    _compile_and_link([(ASAN_FLAGS, output, "_asan")], verbose)
    return output


def build_all(verbose: bool = False) -> None:
    """The library and its host-sanitizer variant, compiled side by side."""
    _compile_and_link([(HIPCC_FLAGS, LIBRARY, ""), (ASAN_FLAGS, ASAN_LIBRARY, "_asan")], verbose)


if __name__ == "__main__":
    if "--asan" in sys.argv:
        print(build_asan(verbose="-v" in sys.argv))
    elif "--all" in sys.argv:
        build_all(verbose="-v" in sys.argv)
    else:
        print(build(verbose="-v" in sys.argv))
