"""Rows so long that the router's kernels would count their columns (float32) or bytes
(bf16: 2^30 columns are 2^31 bytes) past 32 bits are refused, before any HIP call."""
import ctypes

import pytest

from mixture_experts_layer_exclusive_amd import _lib as L

A = 0x10000    # never dereferenced
INV, UNS = L.MOE_ERR_INVALID_ARGUMENT, L.MOE_ERR_UNSUPPORTED
F32, BF16 = L.MOE_DTYPE_F32, L.MOE_DTYPE_BF16


@pytest.mark.parametrize("d,dtype,taken", [(2 ** 25 - 64, BF16, True), (2 ** 25, BF16, False), (2 ** 30, BF16, False),
                                           (2 ** 31 - 64, BF16, False), (2 ** 28, F32, True),
                                           (2 ** 30 + 1, F32, False), (2 ** 31 - 1, F32, False)])
def test_router_rows(d, dtype, taken):
    lib = L.load()
    # (what is taken goes on to the missing ids)
    want = INV if taken else UNS
    g = L.MoeGating(T=2, d=d, dtype=dtype, E=2, k=2, score=0, groups=1, groups_kept=1, group_top=1, renormalise=1, scale=1.0)
    assert lib.moe_route_scored(ctypes.byref(g), A, A, None, A, None, None, A, None, None, 0, None) == want
    p = L.MoeProblem(T=2, d=d, E=2, k=2, f=64, dtype=dtype)
    assert lib.moe_route(ctypes.byref(p), A, A, None, A, None, A, None) == want
