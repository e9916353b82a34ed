"""The grouped products at sizes and in states that the tests of
``test_gpu_grouped`` do not reach, against the same oracle."""
import ctypes

import pytest
import torch

import mixture_experts_layer_exclusive_amd as moe
from grouped_helpers import DEV, check, f64, normal, offsets_of
from mixture_experts_layer_exclusive_amd import _lib as L
from oracle import moe_grouped as G
from test_gpu_grouped import gpu_off, poisoned, ragged

pytestmark = pytest.mark.gpu

# a size whose weight gradient is cut into parts, and so takes a workspace
CUT = dict(rows=21678, E=3, N=1488, K=144)


def test_input_gradient_alone_takes_no_workspace():
    """Only the weight gradient's partial sums use the workspace."""
    R, E, N, K = CUT["rows"], CUT["E"], CUT["N"], CUT["K"]
    need = moe.grouped_workspace_size(2, R, E, N, K, torch.bfloat16)
    assert need > 0
    off = offsets_of(ragged(R, E, seed=3))
    w, dc = normal(1, E, N, K), normal(2, R, N)
    wg, dcg, o = w.to(DEV), dc.to(DEV), gpu_off(off)
    (da, dat), _ = G.matmul_backward(torch.zeros(R, K).numpy(), f64(w), off, f64(dc))
    # the C entry, with no workspace
    out = poisoned(R, K, dtype=torch.bfloat16)
    g = L.MoeGrouped(rows=R, E=E, N=N, K=K, dtype=L.MOE_DTYPE_BF16)
    s = torch.cuda.current_stream()
    assert L.load().moe_grouped_matmul_backward(ctypes.byref(g), None, wg.data_ptr(), o.data_ptr(), dcg.data_ptr(),
                                                out.data_ptr(), None, None, 0, s.cuda_stream) == L.MOE_OK
    torch.cuda.synchronize()
    check(out, da, dat, N, "bf16", "da")
    # the binding allocates none
    out.fill_(3.0e4)
    torch.cuda.synchronize()
    torch.cuda.reset_peak_memory_stats()
    before = torch.cuda.memory_allocated()
    moe.grouped_matmul_backward(None, wg, o, dcg, with_dw=False, out=dict(da=out))
    torch.cuda.synchronize()
    assert torch.cuda.max_memory_allocated() == before
    check(out, da, dat, N, "bf16", "da")
