"""Calls that need more workgroups than one launch takes (its work items are counted in 32
bits) are refused before anything is enqueued. Every call also lacks an output or has two that
overlap, checks that come later: one that gets so far (status 1) was within the limit."""
import ctypes
import os

import pytest

import combine_moe_gate_amd as M
from tests.test_abi import _fake_handle
from tests.test_abi_expert_act import at, no_gpu_only

pytestmark = no_gpu_only
E = 1024  # one row each: a workgroup per expert and column block at least


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(M.LIB_PATH):
        from combine_moe_gate_amd import _build
        _build.build()
    return M.lib()


def handle(s, k=1):
    return _fake_handle(s, E, k, 0, 1 << 24, M.workspace_bytes(s, E, k, 0))


# 1024 rows are 1027 row tiles at most (3 + 1024; 1028 of 256 rows), of 512 threads by 256
# columns: 2^32 - 1 work items hold 8388607 workgroups, so 8168 column blocks (8160 of 1028)
@pytest.mark.parametrize("cols,status", [(8100 * 256, 1), (8192 * 256, 2)])
def test_products(lib, cols, status):
    st = handle(1024)
    assert lib.moe_expert_gemm_act(ctypes.byref(st), at(0), 1, at(1), 8, cols, 1, None, None, None) == status
    half = M.Epilogue(0, 1, None, 0, 0, None, None, None)  # gated: two weight rows a column
    assert lib.moe_expert_gemm_act(ctypes.byref(st), at(0), 1, at(1), 8, cols // 2, 1, ctypes.byref(half), None, None) == status
    assert lib.moe_expert_act_dgrad(ctypes.byref(st), at(0), at(1), cols, 8, 1, None, None) == status
    if status == 2:
        assert "too large for one" in lib.moe_last_error().decode()


def backward(lib, st, n, gb=None, gw=None):
    """With grad_preact in grad_out's place."""
    return lib.moe_expert_act_backward(ctypes.byref(st), at(0), at(1), n, 1, 4, 0, at(2), at(0), 0, gb, gw, None, at(7), 1 << 60, None)


def test_epilogue_backward(lib):
    """256 threads: 16777215 workgroups, 64 of them for clearing rows."""
    st = handle(1024)
    # 1024 rows of 1024 experts are at most 1040 tiles of 64 rows, 512 columns each
    assert backward(lib, st, 16000 * 512) == 1 and backward(lib, st, 16200 * 512) == 2
    # the bias sums take 64 columns of an expert each, the route weights 256 routes
    assert backward(lib, st, 16383 * 64, gb=at(4)) == 1 and backward(lib, st, 16384 * 64, gb=at(4)) == 2
    assert backward(lib, st, 16384 * 64) == 1  # no sums asked for
    assert backward(lib, st, 16383 * 64, gb=at(4), gw=at(5)) == 1
    full = handle(1024 * 16, 16)  # 262144 routes: 1024 workgroups more
    assert backward(lib, full, 16383 * 64, gb=at(4)) == 1 and backward(lib, full, 16383 * 64, gb=at(4), gw=at(5)) == 2


def test_balance_loss_of_many_groups(lib):
    """Its second launch is repeated for the groups past the first: no limit but the rows' count."""
    g = 300000
    args = [at(0), at(1), None, at(2), g, E, 1, g, at(3), at(4), at(5), at(6), None, at(7), 1 << 40, None]
    assert lib.moe_balance_loss(*args) == 1 and "z is NULL" in lib.moe_last_error().decode()


def test_balance_loss_in_one_launch(lib):
    """No workspace where the header says that one launch does."""
    f = lib.moe_balance_workspace_bytes
    for s, e, one in ((32, 1024, True), (33, 1024, False), (1024, 16, True), (1024, 17, False), (1025, 15, False),
                      (33, 496, True), (33, 497, False)):
        assert (f(s, e, 1) == 0) == one, (s, e)
        assert f(s, e, 2) > 0
