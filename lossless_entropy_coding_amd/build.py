"""Build the HIP library libbs.so for gfx950 (in-tree), and the oracle.

Usage: python -m lossless_entropy_coding_amd.build [--asm DIR]
"""
from __future__ import annotations

import argparse
import concurrent.futures
import os
import shutil
import subprocess
import sys
import tempfile

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(HERE, "libbs.so")
ARCH = "gfx950"

SOURCES = ["bs_kernels.hip", "bs_decode.hip", "bs_decode2.hip", "bs_fixed.hip", "bs_fixed_encode.hip", "bs_encode.hip", "bs_noalloc.hip", "bs_kv.hip", "bs_kv_attend.hip", "bs_lora.hip", "bs_kv.cpp", "bs_lora.cpp", "bs_fixed.cpp", "bs_model.cpp", "bs_codec.cpp", "bs_plan.cpp", "bs_stream.cpp",
           "bs_sha256.cpp"]
# packed FP32 instructions are disabled on purpose for every HIP compile
HIP_FLAGS = ["-O3", "-fPIC", "-std=c++17", f"--offload-arch={ARCH}", "-Wall",
             "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
             "-I", CSRC, "-I", INCLUDE]


def hipcc() -> str:
    for cand in (shutil.which("hipcc"), "/opt/rocm/bin/hipcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("hipcc not found")


def build_lib(asm_dir: str | None = None, verbose: bool = False) -> str:
    cc = hipcc()
    with tempfile.TemporaryDirectory() as tmp:
        def compile_one(src: str) -> str:
            obj = os.path.join(tmp, src + ".o")
            cmd = [cc, *HIP_FLAGS, "-c", os.path.join(CSRC, src), "-o", obj]
            if asm_dir and src.endswith(".hip"):
                os.makedirs(asm_dir, exist_ok=True)
                cmd += ["-save-temps=obj"]
                cmd[cmd.index("-o") + 1] = os.path.join(asm_dir, src + ".o")
                obj = os.path.join(asm_dir, src + ".o")
            if verbose:
                print(" ".join(cmd), flush=True)
            r = subprocess.run(cmd, capture_output=True, text=True)
            if r.returncode != 0:
                sys.stderr.write(r.stdout + r.stderr)
                raise RuntimeError(f"compiling {src} failed")
            return obj

        with concurrent.futures.ThreadPoolExecutor(max_workers=min(8, os.cpu_count() or 1)) as pool:
            objs = list(pool.map(compile_one, SOURCES))
        tmp_lib = LIB + ".tmp"
        r = subprocess.run([cc, "-shared", "-fPIC", f"--offload-arch={ARCH}", *objs, "-o", tmp_lib, "-lpthread"],
                           capture_output=True, text=True)
        if r.returncode != 0:
            sys.stderr.write(r.stdout + r.stderr)
            raise RuntimeError("linking libbs.so failed")
        os.replace(tmp_lib, LIB)
    return LIB


def main(argv=None):
    ap = argparse.ArgumentParser()
    ap.add_argument("--asm", default=None, help="keep intermediate files (ISA) in this directory")
    ap.add_argument("-v", action="store_true")
    a = ap.parse_args(argv)
    print(build_lib(a.asm, a.v))


if __name__ == "__main__":
    main()
