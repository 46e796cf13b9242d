"""Build the gfx950 shared library libmoe_gate.so in-tree with hipcc.

    python -m combine_moe_gate_amd._build

hipcc cross-compiles for gfx950 without a GPU present. The same build compiles
tests/c_abi_check, tests/c_abi_ops_check, tests/c_abi_mx4_check and tests/c_abi_mx4_grad_check, C++
programs that drive the library through its C ABI alone.
"""
from __future__ import annotations

import os
import shutil
import subprocess
import sys
import tempfile
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
LIB_NAME = "libmoe_gate.so"
LIB_PATH = os.path.join(HERE, LIB_NAME)
SOURCES = [os.path.join(HERE, "csrc", f) for f in ("api.hip", "gate.hip", "layout.hip", "rows.hip", "gemm.hip", "gemm_bwd.hip",
                                                     "balance.hip", "expert_act.hip", "expert_act_bwd.hip", "mx4.hip", "mx4_act.hip", "mx4_tile.hip", "mx4_stream.hip",
                                                     "mx4_dgrad.hip")]
HEADERS = [os.path.join(HERE, "csrc", f) for f in ("internal.h", "moe_device.h", "gemm_common.h", "ops.h", "expert_act.h", "mx4.h",
                                                     "mx4_product.h")] + [
    os.path.join(ROOT, "include", "moe_gate.h")]

ARCH = "gfx950"
FLAGS = [
    f"--offload-arch={ARCH}",
    "-O3",
    "-std=c++17",
    "-fPIC",
    "-shared",
    # products and sums are rounded separately, as the combine definition states
    "-ffp-contract=off",
    # keep float32 subnormals (the host reference keeps them)
    "-fno-gpu-flush-denormals-to-zero",
    # no packed fp32 arithmetic (v_pk_*_f32) anywhere in the device code
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-Wall",
]


def hipcc() -> str:
    path = shutil.which("hipcc") or "/opt/rocm/bin/hipcc"
    if not os.path.exists(path):
        raise RuntimeError("hipcc not found; the ROCm toolchain is required to build libmoe_gate.so")
    return path


C_CHECKS = [os.path.join(ROOT, "tests", name) for name in ("c_abi_check", "c_abi_ops_check", "c_abi_mx4_check", "c_abi_mx4_grad_check")]


def build_c_checks(verbose: bool = False) -> None:
    """Compile the C++ programs that drive the library through its C ABI alone (GPU tests
    run them). They link LIB_PATH, found next to the binary through its run path."""
    for path in C_CHECKS:
        cmd = [hipcc(), "-O2", "-std=c++17", "-Wall", "-I", os.path.join(ROOT, "include"), path + ".cpp",
               "-L", HERE, "-lmoe_gate", "-Wl,-rpath,$ORIGIN/../combine_moe_gate_amd", "-o", path]
        if verbose:
            print(" ".join(cmd), flush=True)
        res = subprocess.run(cmd, capture_output=True, text=True)
        if res.returncode != 0:
            raise RuntimeError(f"hipcc failed ({res.returncode}):\n{res.stdout}\n{res.stderr}")


def build(verbose: bool = False) -> str:
    """Compile every HIP source, several at a time, into LIB_PATH (always recompiles). Returns the path."""
    tmp = LIB_PATH + ".tmp"
    compile_flags = [f for f in FLAGS if f != "-shared"]

    def run(cmd):
        if verbose:
            print(" ".join(cmd), flush=True)
        res = subprocess.run(cmd, capture_output=True, text=True)
        if res.returncode != 0:
            raise RuntimeError(f"hipcc failed ({res.returncode}):\n{res.stdout}\n{res.stderr}")
        if verbose and res.stderr.strip():
            print(res.stderr, file=sys.stderr)

    with tempfile.TemporaryDirectory() as objects, ThreadPoolExecutor(min(8, os.cpu_count() or 1)) as pool:
        objs = [os.path.join(objects, os.path.basename(s) + ".o") for s in SOURCES]
        list(pool.map(run, [[hipcc(), *compile_flags, "-c", "-I", os.path.join(ROOT, "include"), s, "-o", o]
                            for s, o in zip(SOURCES, objs)]))
        run([hipcc(), *FLAGS, *objs, "-o", tmp])
    os.replace(tmp, LIB_PATH)
    build_c_checks(verbose)
    return LIB_PATH


if __name__ == "__main__":
    print(build(verbose=True))
