"""Build the HIP library libbs.so for gfx950 (in-tree), and the oracle.

Usage: python -m lossless_entropy_coding_amd.build [--asm DIR]
"""
from __future__ import annotations

import argparse
import concurrent.futures
import os
import re
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

SOURCES = ["bs_kernels.hip", "bs_decode.hip", "bs_decode2.hip", "bs_fixed.hip", "bs_fixed_encode.hip", "bs_encode.hip", "bs_noalloc.hip", "bs_kv.hip", "bs_kv_attend.hip", "bs_kv_batch.hip", "bs_kv_shared.hip", "bs_lora.hip", "bs_beam.hip", "bs_kv.cpp", "bs_lora.cpp", "bs_beam.cpp", "bs_fixed.cpp", "bs_model.cpp", "bs_codec.cpp", "bs_plan.cpp", "bs_stream.cpp",
           "bs_sha256.cpp"]
# packed FP32 instructions are disabled on purpose for every HIP compile
HIP_FLAGS = ["-O3", "-fPIC", "-std=c++17", f"--offload-arch={ARCH}", "-Wall",
             "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
             "-I", CSRC, "-I", INCLUDE]


# the compiler's report of each kernel's registers
REPORT = "-Rpass-analysis=kernel-resource-usage"


def check_registers(src: str, report: str, kernels: bool = True) -> None:
    """Raise if a kernel of `src` has accumulation registers (AGPRs).  A matrix
    product's result that is kept in them and read where two blocks join comes
    back stale from this compiler in its later elements, so every kernel's
    launch bounds keep it to 256 registers, where results stay in VGPRs.  Nothing
    else would show that another compiler or a larger kernel has undone it."""
    names = re.findall(r"Function Name: (\S+)", report)
    agprs = [int(n) for n in re.findall(r"\bAGPRs: (\d+)", report)]
    if len(names) != len(agprs) or (kernels and not names):
        raise RuntimeError(f"{src}: the compiler reported {len(agprs)} AGPR counts for {len(names)} kernels")
    used = [f"{k} ({n})" for k, n in zip(names, agprs) if n]
    if used:
        raise RuntimeError(f"{src}: kernels with accumulation registers, in which results can come back stale: {', '.join(used)}")


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
            if src.endswith(".hip"):
                cmd.append(REPORT)
            if verbose:
                print(" ".join(cmd), flush=True)
            r = subprocess.run(cmd, capture_output=True, text=True)
            if r.returncode != 0:
                sys.stderr.write(r.stdout + r.stderr)
                raise RuntimeError(f"compiling {src} failed")
            if src.endswith(".hip"):
                with open(os.path.join(CSRC, src)) as f:
                    check_registers(src, r.stderr, "__global__" in f.read())
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
