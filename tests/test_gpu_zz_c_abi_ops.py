"""The expert products with their epilogue and the router's losses driven from C++ through
the C ABI alone (tests/c_abi_ops_check.cpp), with no Python or PyTorch in the process. It is
compiled with the library by the package build."""
import os
import subprocess

import pytest

pytestmark = pytest.mark.gpu

BIN = os.path.join(os.path.dirname(os.path.abspath(__file__)), "c_abi_ops_check")


def test_c_program_through_the_abi():
    assert os.path.exists(BIN), f"{BIN} is missing: build first (python -m combine_moe_gate_amd._build)"
    print("CASE c_abi_ops_check", flush=True)
    res = subprocess.run([BIN], capture_output=True, text=True, timeout=100)
    print(res.stdout[-2000:], flush=True)
    assert res.returncode == 0, f"exit {res.returncode}\n{res.stdout[-2000:]}\n{res.stderr[-4000:]}"
    assert "c_abi_ops_check: ok" in res.stdout
