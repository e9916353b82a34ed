"""Sizes and workspaces of the grouped products at their limits, on the CPU:
what the entry points accept and refuse before any HIP call."""
import ctypes

import pytest
import torch

from mixture_experts_layer_exclusive_amd import _lib as L

A = 0x10000    # never dereferenced
MIS = 0x10004  # not 16-byte aligned
INV, UNS, WS = L.MOE_ERR_INVALID_ARGUMENT, L.MOE_ERR_UNSUPPORTED, L.MOE_ERR_WORKSPACE_TOO_SMALL


def grp(rows=64, E=8, N=256, K=128, dtype=L.MOE_DTYPE_BF16):
    return L.MoeGrouped(rows=rows, E=E, N=N, K=K, dtype=dtype)


@pytest.fixture(scope="module")
def lib():
    return L.load()


def size(lib, g, op):
    n = ctypes.c_size_t(0)
    return lib.moe_grouped_workspace_size(ctypes.byref(g), op, ctypes.byref(n)), n.value


# one expert whose queue of 100000 rows is cut into parts
CUT = dict(rows=100000, E=1, N=256, K=256)


def test_workspace_of_a_cut_weight_gradient(lib):
    g = grp(**CUT)
    st, n = size(lib, g, L.MOE_GROUPED_OP_BACKWARD)
    assert st == L.MOE_OK and n > 0
    p, back = ctypes.byref(g), lib.moe_grouped_matmul_backward
    for da in (A, None):
        assert back(p, A, A, A, A, da, A, A, n - 1, None) == WS
        assert back(p, A, A, A, A, da, A, None, n, None) == INV
        assert back(p, A, A, A, A, da, A, MIS, n, None) == UNS


@pytest.mark.skipif(torch.cuda.device_count() > 0, reason="the addresses are not memory: nothing may be launched")
def test_calls_that_need_no_workspace_reach_the_launch(lib):
    """With a NULL workspace these pass every check; what stops them here is
    that there is no GPU."""
    p = ctypes.byref(grp(**CUT))
    assert lib.moe_grouped_matmul_backward(p, None, A, A, A, A, None, None, 0, None) == L.MOE_ERR_HIP
    for g in (grp(rows=16, E=1, N=256, K=8192), grp(**CUT)):
        p = ctypes.byref(g)
        assert size(lib, g, L.MOE_GROUPED_OP_MATMUL) == (L.MOE_OK, 0)
        assert size(lib, g, L.MOE_GROUPED_OP_INT8) == (L.MOE_OK, 0)
        assert lib.moe_grouped_matmul(p, A, A, A, A, None, 0, None) == L.MOE_ERR_HIP
        assert lib.moe_grouped_matmul_int8(p, A, A, A, A, A, A, None, 0, None) == L.MOE_ERR_HIP
