"""The grouped products at sizes and in states that the tests of
``test_gpu_grouped`` do not reach, against the same oracle."""
import ctypes

import pytest
import torch

import mixture_experts_layer_exclusive_amd as moe
from grouped_helpers import DEV, TORCH, check, f64, normal, offsets_of
from mixture_experts_layer_exclusive_amd import _lib as L
from oracle import moe_grouped as G
from test_gpu_grouped import (all_outputs, check_int8, graph_state, gpu_off, int8_case, outputs, poisoned, ragged,
                              run_backward, run_matmul)

pytestmark = pytest.mark.gpu

# (op, type, rows, E, N, K).  ``test_grouped_choice`` asserts on the CPU that the
# library's rule takes the kernels that these are here for.
#
# The largest tiles as a stream: more than 512 tiles of ragged queues, so that
# workgroups go on from tile to tile, of 3 slices and more, the last one cut;
# with at most and with more than 8 column tiles, which differ in their order.
STREAMS = [
    ("matmul", "bf16", 12836, 28, 1816, 160),
    ("matmul", "bf16", 7061, 54, 3184, 304),
    ("int8", "bf16", 17286, 48, 1624, 528),
    ("int8", "bf16", 6949, 27, 3272, 592),
    ("int8", "f32", 17596, 7, 1720, 288),
    ("int8", "f32", 11307, 15, 2376, 688),
    ("backward", "bf16", 17044, 34, 240, 1368),
    ("backward", "bf16", 7201, 39, 304, 2744),
]
# Both gradients in one launch, the weight gradient cut into parts, by the
# pairs of tiles that no other test reaches.
JOINT = [
    ("backward", "bf16", 13767, 1, 1024, 24),
    ("backward", "bf16", 765, 1, 72, 40),
    ("backward", "bf16", 16999, 9, 16, 136),
    ("backward", "bf16", 3370, 1, 80, 144),
    ("backward", "f32", 395, 1, 112, 40),
    ("backward", "f32", 487, 1, 36, 72),
    ("backward", "f32", 1997, 2, 2072, 200),
]
# The same by tiles of 128 x 128 in a launch of its own, beside an input gradient
# by the largest tiles.
ALONE = [("backward", "bf16", 34448, 17, 8, 144)]

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


@pytest.mark.parametrize("op,dtype,rows,E,N,K", STREAMS + JOINT + ALONE)
def test_kernels(op, dtype, rows, E, N, K):
    counts = ragged(rows, E, seed=rows)
    what = f"{op} {rows} rows, {E} queues, {N}x{K}"
    if op == "int8":
        # rows before the first queue and behind the last
        qa, sa, qw, sw, off = int8_case(21, counts, N, K, start=3, after=5)
        t = lambda v: torch.from_numpy(v).to(DEV)  # noqa: E731
        c = poisoned(rows + 8, N, dtype=TORCH[dtype])
        moe.grouped_matmul_int8(t(qa), t(sa), t(qw), t(sw), gpu_off(off), out_dtype=TORCH[dtype], c=c)
        check_int8(c, G.matmul_int8(qa, sa, qw, sw, off), dtype, what)
        return
    off = offsets_of(counts, start=3)
    R = rows + 8
    a, w = normal(22, R, K, dtype=dtype), normal(23, E, N, K, dtype=dtype)
    if op == "matmul":
        run_matmul(a, w, off, R, N, dtype, what)
    else:
        run_backward(a, w, off, normal(24, R, N, dtype=dtype), dtype, what)


# The forward, the 8-bit product and both gradients as streams of tiles: rows,
# queues, N, K.
AT_ONCE = (19583, 50, 1160, 1168)


def test_streams_of_every_product_at_once_and_replayed():
    """Two calls of each at once on two streams, and both captured and
    replayed between other work, give the bits of one call alone."""
    rows, E, N, K = AT_ONCE
    states = [graph_state(ragged(rows, E, seed=s), N, K, 80 + s) for s in (1, 2)]
    refs = []
    for st in states:
        all_outputs(*st)
        torch.cuda.synchronize()
        refs.append({key: v.clone() for key, v in outputs(st).items()})

    def clear():
        for st in states:
            for v in outputs(st).values():
                v.zero_()
        torch.cuda.synchronize()

    def compare(what):
        torch.cuda.synchronize()
        for st, ref in zip(states, refs):
            for key, v in outputs(st).items():
                assert torch.equal(v, ref[key]), (what, key)

    streams = [torch.cuda.Stream() for _ in states]
    clear()
    for s, st in zip(streams, states):
        with torch.cuda.stream(s):
            all_outputs(*st)
    compare("two streams")
    graphs = []
    for st in states:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            all_outputs(*st)
        graphs.append(g)
    for it in range(3):
        clear()
        _ = (states[0][0].float() * 2).sum().item()
        for s, g in zip(streams, graphs):
            with torch.cuda.stream(s):
                g.replay()
        compare(f"replay {it}")
