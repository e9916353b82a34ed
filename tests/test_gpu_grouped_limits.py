"""The grouped products at the ends of their documented ranges on the GPU:
the widest matrices, the most rows, and offsets that break the rules at sizes
where workgroups walk many tiles."""
import numpy as np
import pytest
import torch

import mixture_experts_layer_exclusive_amd as moe
from grouped_helpers import DEV, TORCH, normal, offsets_of
from oracle import moe_grouped as G
from test_gpu_grouped import check_int8, gpu_off, int8_case, poisoned, run_backward, run_matmul

pytestmark = pytest.mark.gpu

WIDEST = 1 << 20
MOST_ROWS = 32 * (2 ** 24 - 2 ** 11 - 1)   # of one queue, at N <= 32 and K <= 32


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("wide", ["N", "K"])
@pytest.mark.parametrize("counts", [[3, 0, 2], [70, 300]])
def test_widest_matrices(counts, wide, dtype):
    narrow = 8 if dtype == "bf16" else 4
    N, K = (WIDEST, narrow) if wide == "N" else (narrow, WIDEST)
    off = offsets_of(counts, start=1)
    R, E = int(off[-1]) + 2, len(counts)
    a, w, dc = (normal(i, *s, dtype=dtype) for i, s in enumerate([(R, K), (E, N, K), (R, N)]))
    run_matmul(a, w, off, R, N, dtype)
    if sum(counts) < 10:  # (the oracle's float64 weights and gradients of the others take gigabytes)
        run_backward(a, w, off, dc, dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_widest_int8_outputs(dtype):
    qa, sa, qw, sw, off = int8_case(5, [3, 0, 40], WIDEST, 16, start=1, after=2)
    t = lambda v: torch.from_numpy(v).to(DEV)  # noqa: E731
    c = poisoned(qa.shape[0], WIDEST, dtype=TORCH[dtype])
    moe.grouped_matmul_int8(t(qa), t(sa), t(qw), t(sw), gpu_off(off), out_dtype=TORCH[dtype], c=c)
    check_int8(c, G.matmul_int8(qa, sa, qw, sw, off), dtype)


def test_most_rows():
    """More than 2^32 elements of a and of c, in one queue but for a few rows.
    Small integers, so every sum is exact in float32 and in bf16; compared on
    the GPU in pieces, and in float64 at picked rows."""
    R, N, K = MOST_ROWS - 2 * 31, 8, 8   # (three queues begin a row tile each)
    first = 5
    off = torch.tensor([first, first, R - 3, R], dtype=torch.int32, device=DEV)
    g = torch.Generator(device=DEV).manual_seed(7)
    a = torch.empty(R, K, dtype=torch.int8, device=DEV)
    step = 1 << 26
    for r in range(0, R, step):
        a[r:r + step] = torch.randint(-2, 3, (min(step, R - r), K), generator=g, device=DEV, dtype=torch.int8)
    w = torch.randint(-2, 3, (3, N, K), generator=g, device=DEV, dtype=torch.int8)
    ab = a.to(torch.bfloat16)
    wb = w.to(torch.bfloat16)
    c = torch.full((R, N), 99.0, dtype=torch.bfloat16, device=DEV)
    moe.grouped_matmul(ab, wb, off, c=c)

    def compare(got, src, mats):
        assert (got[:first] == 99).all()
        for lo, hi, e in ((first, R - 3, 1), (R - 3, R, 2)):
            for r in range(lo, hi, step):
                s = slice(r, min(r + step, hi))
                want = (src[s].float() @ mats[e].float().t()).to(torch.bfloat16)
                assert torch.equal(got[s], want), (r, e)
        pick = torch.tensor([first, 2 ** 28 - 1, 2 ** 28, 2 ** 29 - 2 ** 17, R - 4], device=DEV)
        assert torch.equal(got[pick].double(), src[pick].double() @ mats[1].double().t())

    compare(c, ab, wb)
    c.fill_(99.0)
    g = moe.grouped_matmul_backward(None, wb, off, ab, with_dw=False, out=dict(da=c))
    compare(g["da"], ab, wb.transpose(1, 2).contiguous())


def test_most_rows_int8():
    R, N, K = MOST_ROWS, 8, 16
    g = torch.Generator(device=DEV).manual_seed(8)
    a = torch.empty(R, K, dtype=torch.int8, device=DEV)
    step = 1 << 26
    for r in range(0, R, step):
        a[r:r + step] = torch.randint(-2, 3, (min(step, R - r), K), generator=g, device=DEV, dtype=torch.int8)
    w = torch.randint(-2, 3, (N, K), generator=g, device=DEV, dtype=torch.int8)
    sa, sw = torch.ones(R, device=DEV), torch.full((N,), 0.5, device=DEV)
    sa[-1] = 4.0
    c = moe.grouped_matmul_int8(a, sa, w, sw)
    for r in range(0, R, step):
        s = slice(r, min(r + step, R))
        # (halves of whole numbers up to 64: exact in bf16)
        want = ((a[s].float() @ w.float().t()) * sa[s, None] * 0.5).to(torch.bfloat16)
        assert torch.equal(c[s], want), r


@pytest.mark.parametrize("kind", ["shuffled", "up and down", "beyond"])
def test_offsets_that_break_the_rules_at_stream_sizes(kind):
    """Queues that overlap, descend or lie outside: any values in the outputs,
    but nothing around them is written, nor a row that no queue can hold."""
    R, E, N, K = 9000, 40, 1272, 1040
    rng = np.random.default_rng(3)
    if kind == "shuffled":
        vals = rng.integers(0, R + 1, E + 1)
    elif kind == "up and down":
        vals = np.where(np.arange(E + 1) % 2 == 0, 17, R)
    else:
        vals = rng.integers(-2 ** 31, 2 ** 31, E + 1)
    o = torch.from_numpy(vals.astype(np.int64)).to(torch.int32).to(DEV)
    pad = 1 << 16

    def guarded(*shape, dtype):
        n = int(np.prod(shape))
        buf = torch.full((n + 2 * pad,), 7.0, dtype=dtype, device=DEV)
        return buf[pad:pad + n].view(shape), lambda: (buf[:pad] == 7).all() and (buf[pad + n:] == 7).all()
    for dt in (torch.bfloat16, torch.float32):
        a, w = torch.ones(R, K, dtype=dt, device=DEV), torch.ones(E, N, K, dtype=dt, device=DEV)
        c, c_ok = guarded(R, N, dtype=dt)
        da, da_ok = guarded(R, K, dtype=dt)
        dw, dw_ok = guarded(E, N, K, dtype=dt)
        c8, c8_ok = guarded(R, N, dtype=dt)
        moe.grouped_matmul(a, w, o, c=c)
        moe.grouped_matmul_backward(a, w, o, torch.ones(R, N, dtype=dt, device=DEV), out=dict(da=da, dw=dw))
        moe.grouped_matmul_int8(a.to(torch.int8), torch.ones(R, device=DEV), w.to(torch.int8),
                                torch.ones(E, N, device=DEV), o, out_dtype=dt, c=c8)
        torch.cuda.synchronize()
        assert c_ok() and da_ok() and dw_ok() and c8_ok()
        if kind == "up and down":
            for out in (c, da, c8):
                assert (out[:17] == 7).all()
