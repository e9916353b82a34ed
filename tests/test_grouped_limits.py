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


# The most rows of one queue at the least width: one 32-row tile counts for
# each 32 rows begun, and there may be fewer than 2^24 - 2^11 of them.
MOST_ROWS = 32 * (2 ** 24 - 2 ** 11 - 1)


@pytest.mark.parametrize("op", [1, 2, 3])
@pytest.mark.parametrize("dtype", [L.MOE_DTYPE_BF16, L.MOE_DTYPE_F32])
def test_the_most_rows(lib, op, dtype):
    kw = dict(E=1, N=8, K=16 if op == 3 else 8, dtype=dtype)
    assert size(lib, grp(rows=MOST_ROWS, **kw), op)[0] == L.MOE_OK
    assert size(lib, grp(rows=MOST_ROWS + 1, **kw), op)[0] == UNS
    # as many tiles in two columns
    half = 32 * ((2 ** 24 - 2 ** 11) // 2 - 1)
    kw["N"] = 40
    assert size(lib, grp(rows=half, **kw), op)[0] == L.MOE_OK
    assert size(lib, grp(rows=half + 1, **kw), op)[0] == UNS


@pytest.mark.parametrize("rows", [2 ** 29, 2 ** 31 - 2 ** 16, 2 ** 31 - 2 ** 16 + 1, 2 ** 62, 2 ** 63 - 1])
def test_more_rows_are_refused(lib, rows):
    for op in (1, 2, 3):
        for kw in (dict(N=8, K=16), dict(N=1 << 20, K=1 << 20)):
            assert size(lib, grp(rows=rows, E=1, **kw), op)[0] == UNS


@pytest.mark.parametrize("E", [1, 3, 256])
def test_what_always_fits(lib, E):
    """rows * max(N, K, 32) and E * N * K up to 2^32."""
    for width in (16, 40, 64, 1000, 4096, 1 << 20):
        rows = 2 ** 32 // max(width, 32)
        for N, K in ((width, 16), (16, width)):
            for dtype in (L.MOE_DTYPE_BF16, L.MOE_DTYPE_F32):
                for op in (1, 2):
                    assert size(lib, grp(rows=rows, E=E, N=N, K=K, dtype=dtype), op)[0] == L.MOE_OK, (rows, N, K)
