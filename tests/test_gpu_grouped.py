"""The grouped products and the 8-bit integer product on the GPU, against the
float64 oracle (``oracle.moe_grouped``), element by element.

Bounds are derived, not tuned: see ``grouped_helpers.check`` for the float
products.  The integer product's sum is exact, so its result carries the
roundings of float(sum), of the two scalings (2^-24 each) and of the output
type.  Codes and scales of the quantisation are compared bit for bit.
Outputs are filled with a mark before each call, so an unwritten element, or
a row written outside the queues, fails.
"""
import numpy as np
import pytest
import torch

import mixture_experts_layer_exclusive_amd as moe
from grouped_helpers import DEV, QUEUES, TORCH, check, f64, normal, offsets_of
from oracle import moe_grouped as G

pytestmark = pytest.mark.gpu

# (N, K): the shortest rows, widths around the tiles' edges, widths that no
# tile divides, long reductions
WIDTHS = [(8, 8), (64, 128), (72, 40), (136, 264), (256, 1032), (520, 64), (1000, 520)]
LARGE = {
    # enough rows and columns for the largest tiles, ragged in every size
    "ragged": ([1900, 0, 1, 2500, 300, 3491], 2056, 520),
    "one queue": ([4100], 4104, 200),
}


def gpu_off(off):
    return torch.from_numpy(off).to(DEV)


def poisoned(*shape, dtype):
    return torch.full(shape, 3.0e4, dtype=dtype, device=DEV)


def ws_for(op, R, E, N, K, dtype):
    """A workspace of exactly the stated size, filled with NaN patterns, with
    a guard behind it."""
    n = moe.grouped_workspace_size(op, R, E, N, K, dtype)
    if n == 0:
        return None, lambda: None
    buf = torch.full((n + 4096,), 0xFF, dtype=torch.uint8, device=DEV)

    def guard():
        assert (buf[n:] == 0xFF).all(), "written past the workspace"
    return buf[:n], guard


def run_matmul(a, w, off, R, N, dtype, what=""):
    E, _, K = w.shape
    c = poisoned(R, N, dtype=TORCH[dtype])
    ws, guard = ws_for(1, R, E, N, K, TORCH[dtype])
    moe.grouped_matmul(a.to(DEV), w.to(DEV), gpu_off(off), c=c, ws=ws)
    torch.cuda.synchronize()
    guard()
    ref, terms = G.matmul(f64(a), f64(w), off)
    check(c, ref, terms, K, dtype, what)
    out = np.isnan(ref)
    assert (f64(c)[out] == f64(poisoned(1, dtype=TORCH[dtype]))[0]).all(), "a row outside the queues was written"
    return c


def run_backward(a, w, off, dc, dtype, what=""):
    E, N, K = w.shape
    R = a.shape[0]
    out = dict(da=poisoned(R, K, dtype=TORCH[dtype]), dw=poisoned(E, N, K, dtype=TORCH[dtype]))
    ws, guard = ws_for(2, R, E, N, K, TORCH[dtype])
    g = moe.grouped_matmul_backward(a.to(DEV), w.to(DEV), gpu_off(off), dc.to(DEV), out=out, ws=ws)
    torch.cuda.synchronize()
    guard()
    (da, dat), (dw, dwt) = G.matmul_backward(f64(a), f64(w), off, f64(dc))
    check(g["da"], da, dat, N, dtype, what + " da")
    longest = max([hi - lo for _, lo, hi in G.queues(off)] + [1])
    check(g["dw"], dw, dwt, longest, dtype, what + " dw")
    if R:
        outside = np.isnan(da)
        assert (f64(g["da"])[outside] == f64(poisoned(1, dtype=TORCH[dtype]))[0]).all()
    return g


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("N,K", WIDTHS)
@pytest.mark.parametrize("queues", list(QUEUES))
def test_matmul(queues, N, K, dtype):
    counts = QUEUES[queues]
    if len(counts) * N * K > 4e7:
        N, K = min(N, 136), min(K, 264)
    off = offsets_of(counts, start=3)
    R = int(off[-1]) + 5  # rows before the first and behind the last queue
    a, w = normal(1, R, K, dtype=dtype), normal(2, len(counts), N, K, dtype=dtype)
    run_matmul(a, w, off, R, N, dtype, what=f"{queues} {N}x{K}")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("N,K", WIDTHS)
@pytest.mark.parametrize("queues", list(QUEUES))
def test_backward(queues, N, K, dtype):
    counts = QUEUES[queues]
    if len(counts) * N * K > 4e7:
        N, K = min(N, 136), min(K, 264)
    off = offsets_of(counts, start=3)
    R = int(off[-1]) + 5
    a, w = normal(3, R, K, dtype=dtype), normal(4, len(counts), N, K, dtype=dtype)
    dc = normal(5, R, N, dtype=dtype)
    run_backward(a, w, off, dc, dtype, what=f"{queues} {N}x{K}")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("name", list(LARGE))
def test_large(name, dtype):
    counts, N, K = LARGE[name]
    off = offsets_of(counts, start=1)
    R = int(off[-1]) + 9
    a, w = normal(6, R, K, dtype=dtype), normal(7, len(counts), N, K, dtype=dtype)
    run_matmul(a, w, off, R, N, dtype, what=name)
    run_matmul(normal(8, R, N, dtype=dtype), normal(9, len(counts), K, N, dtype=dtype), off, R, K, dtype, what=name)
    run_backward(a, w, off, normal(10, R, N, dtype=dtype), dtype, what=name)


def test_no_rows():
    w = normal(1, 3, 64, 64).to(DEV)
    off = torch.zeros(4, dtype=torch.int32, device=DEV)
    a = torch.empty(0, 64, dtype=torch.bfloat16, device=DEV)
    assert moe.grouped_matmul(a, w, off).shape == (0, 64)
    g = moe.grouped_matmul_backward(a, w, off, a, out=dict(dw=poisoned(3, 64, 64, dtype=torch.bfloat16)))
    assert g["da"].shape == (0, 64) and (g["dw"] == 0).all()
    codes, scales = moe.quantize_rows_int8(a)
    assert codes.shape == (0, 64) and scales.shape == (0,)
    c = moe.grouped_matmul_int8(codes, scales, w.to(torch.int8), torch.ones(3, 64, device=DEV), off)
    assert c.shape == (0, 64)


def test_one_gradient_at_a_time():
    counts, N, K = [5, 0, 130], 136, 72
    off = offsets_of(counts)
    a, w, dc = (normal(i, *s).to(DEV) for i, s in enumerate([(135, K), (3, N, K), (135, N)]))
    o = gpu_off(off)
    both = moe.grouped_matmul_backward(a, w, o, dc)
    da = moe.grouped_matmul_backward(None, w, o, dc, with_dw=False)
    dw = moe.grouped_matmul_backward(a, None, o, dc, with_da=False)
    assert da["dw"] is None and dw["da"] is None
    assert torch.equal(da["da"], both["da"]) and torch.equal(dw["dw"], both["dw"])


def test_gradients_against_differences():
    """The product is bilinear, so a central difference of the loss along a
    direction equals the gradient's projection up to float32 rounding."""
    counts, N, K = [20, 0, 45], 36, 52
    off = offsets_of(counts)
    o = gpu_off(off)
    a, w, dc, u, v = (normal(i, *s, dtype="f32").to(DEV)
                      for i, s in enumerate([(65, K), (3, N, K), (65, N), (65, K), (3, N, K)]))
    g = moe.grouped_matmul_backward(a, w, o, dc)
    loss = lambda a_, w_: (moe.grouped_matmul(a_, w_, o).double() * dc.double()).sum().item()  # noqa: E731
    for got, dirn, lo, hi in ((g["da"], u, (a - u, w), (a + u, w)), (g["dw"], v, (a, w - v), (a, w + v))):
        want = (got.double() * dirn.double()).sum().item()
        have = (loss(*hi) - loss(*lo)) / 2
        # each loss sums 65 * 36 values, each of 52 terms of size about
        # sqrt(2); errors of 2 * 53 * 2^-24 of the absolute sum, added up
        bound = 4 * 53 * 2.0 ** -24 * 65 * N * K * 2.0 * 2.0 ** 0.5
        assert abs(want - have) <= bound, (want, have, bound)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_special_values_stay_in_their_rows(dtype, bad):
    """A row's NaN or infinity reaches that row's results only: not those of
    its neighbours, whose tails and padding share tiles with it."""
    counts, N, K = [3, 40, 0, 70], 136, 72
    off = offsets_of(counts)
    o = gpu_off(off)
    R = int(off[-1])
    a, w, dc = (normal(i, *s, dtype=dtype).to(DEV) for i, s in enumerate([(R, K), (4, N, K), (R, N)]))
    row = 10  # in queue 1
    c0 = moe.grouped_matmul(a, w, o)
    g0 = moe.grouped_matmul_backward(a, w, o, dc)
    a1, dc1 = a.clone(), dc.clone()
    a1[row] = bad
    dc1[row] = bad
    c1 = moe.grouped_matmul(a1, w, o)
    g1 = moe.grouped_matmul_backward(a1, w, o, dc1)
    keep = torch.arange(R, device=DEV) != row
    assert torch.equal(c1[keep], c0[keep]) and not torch.isfinite(c1[row]).any()
    assert torch.equal(g1["da"][keep], g0["da"][keep]) and not torch.isfinite(g1["da"][row]).any()
    others = [0, 2, 3]
    assert torch.equal(g1["dw"][others], g0["dw"][others]) and not torch.isfinite(g1["dw"][1]).any()
    # an expert's weights reach its own rows only
    w1 = w.clone()
    w1[1] = bad
    c2 = moe.grouped_matmul(a, w1, o)
    outside = torch.ones(R, dtype=torch.bool, device=DEV)
    outside[int(off[1]):int(off[2])] = False
    assert torch.equal(c2[outside], c0[outside]) and not torch.isfinite(c2[~outside]).any()
    d2 = moe.grouped_matmul_backward(a, w1, o, dc, with_dw=False)["da"]
    assert torch.equal(d2[outside], g0["da"][outside]) and not torch.isfinite(d2[~outside]).any()
    # one output channel's weights reach that channel only
    w1 = w.clone()
    w1[:, 7] = bad
    c3 = moe.grouped_matmul(a, w1, o)
    cols = torch.arange(N, device=DEV) != 7
    assert torch.equal(c3[:, cols], c0[:, cols]) and not torch.isfinite(c3[:, 7]).any()
    # a column of a or dc reaches that column of dw only
    a2 = a.clone()
    a2[:, 5] = bad
    d3 = moe.grouped_matmul_backward(a2, None, o, dc, with_da=False)["dw"]
    kc = torch.arange(K, device=DEV) != 5
    assert torch.equal(d3[:, :, kc], g0["dw"][:, :, kc]) and not torch.isfinite(d3[[0, 1, 3], :, 5]).any()


def ragged(total, E, seed):
    """E queue lengths that sum to total: a third of the queues empty, the
    others uneven, with a queue of one row."""
    rng = np.random.default_rng(seed)
    share = rng.random(E) ** 2 * (rng.random(E) > 1 / 3)
    share[rng.integers(E)] = 1.0
    counts = np.floor(share / share.sum() * total).astype(int)
    counts[np.argmax(counts)] += total - counts.sum()
    if E > 2 and (counts == 0).any():
        counts[np.argmax(counts)] -= 1
        counts[np.argmin(counts)] += 1
    return [int(v) for v in counts]


# Sizes at which the choice of the kernel falls on the less usual ones: the
# 64 x 64 split tiles; the largest tiles as one stream of one, two, three and
# many slices per tile, several tiles per workgroup; queues cut into parts.
CHOICES = [
    ("matmul", "bf16", 1370, 1, 496, 1744),
    ("matmul", "bf16", 12626, 100, 464, 16),
    ("matmul", "bf16", 5000, 3, 2056, 1160),
    ("backward", "bf16", 1072, 8, 2704, 512),
    ("backward", "bf16", 5241, 8, 176, 1728),
    ("backward", "bf16", 8947, 40, 48, 3232),
    ("backward", "bf16", 21678, 3, 1488, 144),
    ("backward", "bf16", 35168, 5, 528, 336),
    ("backward", "bf16", 3061, 16, 3600, 464),
    ("backward", "bf16", 56000, 40, 304, 520),
    ("backward", "bf16", 9000, 34, 1272, 2040),
    ("backward", "f32", 3061, 16, 3600, 464),
    ("backward", "f32", 13, 1, 3536, 4144),
    ("backward", "f32", 15230, 3, 128, 1536),
    ("backward", "f32", 10969, 3, 2608, 144),
    ("int8", "bf16", 1427, 2, 480, 4176),
    ("int8", "bf16", 9537, 8, 944, 32),
    ("int8", "f32", 865, 3, 1008, 3920),
    ("int8", "f32", 13787, 3, 592, 528),
]


@pytest.mark.parametrize("op,dtype,rows,E,N,K", CHOICES)
def test_each_kernel(op, dtype, rows, E, N, K):
    counts = ragged(rows, E, seed=rows)
    assert sum(counts) == rows and min(counts) >= 0
    what = f"{op} {rows} rows, {E} queues, {N}x{K}"
    if op == "int8":
        qa, sa, qw, sw, off = int8_case(16, counts, N, K)
        t = lambda v: torch.from_numpy(v).to(DEV)  # noqa: E731
        c = poisoned(rows, N, dtype=TORCH[dtype])
        moe.grouped_matmul_int8(t(qa), t(sa), t(qw), t(sw), gpu_off(off), out_dtype=TORCH[dtype], c=c)
        check_int8(c, G.matmul_int8(qa, sa, qw, sw, off), dtype, what)
        return
    off = offsets_of(counts)
    a, w = normal(17, rows, K, dtype=dtype), normal(18, E, N, K, dtype=dtype)
    if op == "matmul":
        run_matmul(a, w, off, rows, N, dtype, what)
    else:
        run_backward(a, w, off, normal(19, rows, N, dtype=dtype), dtype, what)


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_special_values_stay_in_their_rows_of_a_stream_of_tiles(bad):
    """As above, at sizes where a workgroup goes from tile to tile: the rows
    behind a queue, the end of the reduction and the next tile's first slice
    lie in LDS beside one another."""
    # forward: one quarter-full slice per tile
    rows, E, N, K = 12626, 100, 464, 16
    off = offsets_of(ragged(rows, E, seed=rows))
    o = gpu_off(off)
    a, w = normal(1, rows, K).to(DEV), normal(2, E, N, K).to(DEV)
    e = int(np.argmax(np.diff(off)))
    row = int(off[e]) + 3
    c0 = moe.grouped_matmul(a, w, o)
    a1, w1 = a.clone(), w.clone()
    a1[row] = bad
    c1 = moe.grouped_matmul(a1, w, o)
    keep = torch.arange(rows, device=DEV) != row
    assert torch.equal(c1[keep], c0[keep]) and not torch.isfinite(c1[row]).any()
    w1[e] = bad
    c2 = moe.grouped_matmul(a, w1, o)
    keep = torch.ones(rows, dtype=torch.bool, device=DEV)
    keep[int(off[e]):int(off[e + 1])] = False
    assert torch.equal(c2[keep], c0[keep]) and not torch.isfinite(c2[~keep]).any()
    # input gradient: three slices, the last not full
    rows, E, N, K = 5241, 8, 176, 1728
    off = offsets_of(ragged(rows, E, seed=rows))
    o = gpu_off(off)
    dc, w = normal(3, rows, N).to(DEV), normal(4, E, N, K).to(DEV)
    e = int(np.argmax(np.diff(off)))
    d0 = moe.grouped_matmul_backward(None, w, o, dc, with_dw=False)["da"]
    w1 = w.clone()
    w1[e] = bad
    keep = torch.ones(rows, dtype=torch.bool, device=DEV)
    keep[int(off[e]):int(off[e + 1])] = False
    d1 = moe.grouped_matmul_backward(None, w1, o, dc, with_dw=False)["da"]
    assert torch.equal(d1[keep], d0[keep]) and not torch.isfinite(d1[~keep]).any()
    # weight gradient in parts: a row reaches its own expert only
    rows, E, N, K = 21678, 3, 1488, 144
    off = offsets_of([9000, 0, 12678])
    o = gpu_off(off)
    a, dc = normal(5, rows, K).to(DEV), normal(6, rows, N).to(DEV)
    g0 = moe.grouped_matmul_backward(a, None, o, dc, with_da=False)["dw"]
    for row, hit in ((8999, 0), (9000, 2)):
        dc1 = dc.clone()
        dc1[row] = bad
        g1 = moe.grouped_matmul_backward(a, None, o, dc1, with_da=False)["dw"]
        others = [i for i in range(E) if i != hit]
        assert torch.equal(g1[others], g0[others]) and not torch.isfinite(g1[hit]).any()


def test_offsets_outside_the_matrix_stay_inside_the_arrays():
    """Offsets that break the rules (beyond the rows, negative, descending)
    give unspecified values, but nothing outside the outputs is written."""
    R, E, N, K = 100, 4, 72, 40
    for vals in ([0, 50, 400, 90, 2 ** 31 - 1], [-5, 10, 5, 200, 100], [2 ** 31 - 1] * 5, [-2 ** 31] * 5):
        o = torch.tensor(vals, dtype=torch.int64).to(torch.int32).to(DEV)
        for dt in (torch.bfloat16, torch.float32):
            buf = torch.full((R * N + 2 * 4096,), 7.0, dtype=dt, device=DEV)
            c = buf[4096:4096 + R * N].view(R, N)
            a, w = torch.ones(R, K, dtype=dt, device=DEV), torch.ones(E, N, K, dtype=dt, device=DEV)
            moe.grouped_matmul(a, w, o, c=c)
            bda = torch.full((R * K + 2 * 4096,), 7.0, dtype=dt, device=DEV)
            bdw = torch.full((E * N * K + 2 * 4096,), 7.0, dtype=dt, device=DEV)
            moe.grouped_matmul_backward(a, w, o, c, out=dict(da=bda[4096:4096 + R * K].view(R, K),
                                                             dw=bdw[4096:4096 + E * N * K].view(E, N, K)))
            torch.cuda.synchronize()
            for b, n in ((buf, R * N), (bda, R * K), (bdw, E * N * K)):
                assert (b[:4096] == 7).all() and (b[4096 + n:] == 7).all()


# ---- 8-bit integers -----------------------------------------------------------

def int8_case(seed, counts, N, K, start=0, after=0):
    rng = np.random.default_rng(seed)
    off = offsets_of(counts, start)
    R, E = int(off[-1]) + after, len(counts)
    qa = rng.integers(-127, 128, (R, K)).astype(np.int8)
    qw = rng.integers(-127, 128, (E, N, K)).astype(np.int8)
    # extreme codes: the largest sums, of one sign
    qa[R // 2:R // 2 + 1], qw[:, N // 2] = -128, -128
    qa[R // 3:R // 3 + 1], qw[:, N // 3] = 127, 127
    sa = (rng.random(R) + 0.5).astype(np.float32) * np.float32(2.0) ** rng.integers(-20, 20, R).astype(np.float32)
    sw = (rng.random((E, N)) + 0.5).astype(np.float32)
    return qa, sa, qw, sw, off


def check_int8(c, ref, dtype, what=""):
    got = f64(c)
    have = ~np.isnan(ref)
    step = 4 * 2.0 ** -24 + (2.0 ** -8 if dtype == "bf16" else 0.0)
    assert (np.abs(got - ref)[have] <= step * (1 + 2.0 ** -8) * np.abs(ref[have])).all(), what
    assert (got[~have] == f64(poisoned(1, dtype=TORCH[dtype]))[0]).all(), "a row outside the queues was written"


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("N,K", [(8, 16), (64, 128), (72, 48), (136, 272), (256, 1040), (520, 64), (1000, 528)])
@pytest.mark.parametrize("queues", list(QUEUES))
def test_int8(queues, N, K, dtype):
    counts = QUEUES[queues]
    if len(counts) * N * K > 4e7:
        N, K = min(N, 136), min(K, 272)
    qa, sa, qw, sw, off = int8_case(11, counts, N, K, start=3, after=5)
    R, E = qa.shape[0], len(counts)
    c = poisoned(R, N, dtype=TORCH[dtype])
    ws, guard = ws_for(3, R, E, N, K, TORCH[dtype])
    t = lambda v: torch.from_numpy(v).to(DEV)  # noqa: E731
    moe.grouped_matmul_int8(t(qa), t(sa), t(qw), t(sw), gpu_off(off), out_dtype=TORCH[dtype], c=c, ws=ws)
    torch.cuda.synchronize()
    guard()
    check_int8(c, G.matmul_int8(qa, sa, qw, sw, off), dtype, f"{queues} {N}x{K}")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("R,N,K", [(1, 8, 16), (1, 4096, 2048), (16, 1000, 8208), (33, 136, 131056), (300, 520, 4096),
                                   (4100, 2056, 528)])
def test_int8_dense(R, N, K, dtype):
    qa, sa, qw, sw, off = int8_case(12, [R], N, K)
    c = poisoned(R, N, dtype=TORCH[dtype])
    ws, guard = ws_for(3, R, 1, N, K, TORCH[dtype])
    t = lambda v: torch.from_numpy(v).to(DEV)  # noqa: E731
    moe.grouped_matmul_int8(t(qa), t(sa), t(qw[0]), t(sw[0]), out_dtype=TORCH[dtype], c=c, ws=ws)
    torch.cuda.synchronize()
    guard()
    check_int8(c, G.matmul_int8(qa, sa, qw, sw, off), dtype)


def test_int8_large():
    counts, N, K = LARGE["ragged"][0], 2056, 528
    qa, sa, qw, sw, off = int8_case(13, counts, N, K, start=1, after=9)
    t = lambda v: torch.from_numpy(v).to(DEV)  # noqa: E731
    for dtype in ("bf16", "f32"):
        c = poisoned(qa.shape[0], N, dtype=TORCH[dtype])
        moe.grouped_matmul_int8(t(qa), t(sa), t(qw), t(sw), gpu_off(off), out_dtype=TORCH[dtype], c=c)
        check_int8(c, G.matmul_int8(qa, sa, qw, sw, off), dtype)


def test_int8_nan_scales_poison_their_row_and_channel():
    qa, sa, qw, sw, off = int8_case(14, [40, 30], 72, 48)
    sa[7], sw[1, 5] = np.nan, np.nan
    t = lambda v: torch.from_numpy(v).to(DEV)  # noqa: E731
    c = f64(moe.grouped_matmul_int8(t(qa), t(sa), t(qw), t(sw), gpu_off(off)))
    want = np.zeros(c.shape, bool)
    want[7] = True
    want[40:, 5] = True
    assert np.array_equal(np.isnan(c), want)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,cols", [(1, 16), (9, 16), (64, 48), (5, 1040), (33, 2048), (7, 4112), (3, 16400), (2, 70000)])
def test_quantize_rows_bit_exact(rows, cols, dtype):
    rng = np.random.default_rng(rows * 1000 + cols)
    x = rng.standard_normal((rows, cols)).astype(np.float32)
    x *= np.exp2(rng.integers(-60, 60, (rows, 1))).astype(np.float32)
    if rows > 4:
        x[0] = 0
        x[1] = -0.0
        x[2, :] = rng.integers(-254, 255, cols) / 2   # scale 1 with ties
        x[2, 0] = 127
        x[3] = np.exp2(-149.0) * rng.integers(-100, 101, cols)   # subnormals
        x[4, cols // 2] = np.inf
    if rows > 5:
        x[5, cols - 1] = np.nan
        x[6] = 0
        x[6, cols - 1] = -np.finfo(np.float32).max / 2
    t = torch.from_numpy(x).to(TORCH[dtype])
    codes = torch.full((rows, cols), 99, dtype=torch.int8, device=DEV)
    scales = torch.full((rows,), -1.0, device=DEV)
    moe.quantize_rows_int8(t.to(DEV), codes=codes, scales=scales)
    q, s = G.quantize_rows_int8(t.float().numpy())
    assert np.array_equal(np.isnan(scales.cpu().numpy()), np.isnan(s))
    fine = ~np.isnan(s)
    assert np.array_equal(scales.cpu().numpy()[fine].view(np.uint32), s[fine].view(np.uint32))
    assert np.array_equal(codes.cpu().numpy(), q)


# ---- how they are used ----------------------------------------------------------

def layer(seed=31, T=700, d=256, E=16, k=4, f=384, dtype="bf16"):
    ids_seed = torch.Generator().manual_seed(seed)
    x = normal(seed, T, d, dtype=dtype)
    logits = torch.randn(T, E, generator=ids_seed)
    w1 = normal(seed + 1, E, f, d, dtype=dtype, scale=d ** -0.5)
    w2 = normal(seed + 2, E, d, f, dtype=dtype, scale=f ** -0.5)
    dy = normal(seed + 3, T, d, dtype=dtype)
    return x, logits, w1, w2, dy


def test_layer_of_squared_relu_experts_with_its_gradients():
    """route, dispatch, two grouped products with another activation between
    them, combine; then the gradients through both.  Against torch's double
    precision on the same routing; every step that rounds to bf16 is off by
    2^-8 relative at most, and the chain has five such steps (h, the square,
    y_perm, y, or their gradients), so the relative 2-norm stays under
    5 * 2^-8."""
    x, logits, w1, w2, dy = layer()
    T, d = x.shape
    E, k = w1.shape[0], 4
    xg, w1g, w2g, dyg = (v.to(DEV) for v in (x, w1, w2, dy))
    ids, gates, _ = moe.route(k, logits=logits.to(DEV))
    q = moe.dispatch(ids, E, x=xg, with_x_perm=True)
    off, xp = q["offsets"], q["x_perm"]
    h = moe.grouped_matmul(xp, w1g, off)
    act = torch.relu(h).square()
    yp = moe.grouped_matmul(act, w2g, off)
    y = moe.combine(yp, q["assign_pos"], gates)
    # backward: each queue row's dy, weighted by its gate
    tok = torch.div(q["sorted_assign"].long(), k, rounding_mode="floor")
    dyp = (dyg[tok].float() * gates.reshape(-1)[q["sorted_assign"].long()][:, None]).to(torch.bfloat16)
    g2 = moe.grouped_matmul_backward(act, w2g, off, dyp)
    dh = (g2["da"].float() * 2 * torch.relu(h).float()).to(torch.bfloat16)
    g1 = moe.grouped_matmul_backward(xp, w1g, off, dh)
    dx = moe.combine(g1["da"], q["assign_pos"], torch.ones_like(gates))

    xd, w1d, w2d = (v.double().clone().requires_grad_() for v in (x, w1, w2))
    gd, idc = gates.double().cpu(), ids.cpu().long()
    yd = torch.zeros(T, d, dtype=torch.float64)
    for e in range(E):
        t_, j_ = torch.where(idc == e)
        ye = torch.relu(xd[t_] @ w1d[e].T).square() @ w2d[e].T
        yd = yd.index_add(0, t_, ye * gd[t_, j_][:, None])
    yd.backward(dy.double())
    rel = lambda a, b: (torch.linalg.norm(a.double().cpu() - b) / torch.linalg.norm(b)).item()  # noqa: E731
    for got, ref, name in ((y, yd.detach(), "y"), (dx, xd.grad, "dx"), (g1["dw"], w1d.grad, "dw1"),
                           (g2["dw"], w2d.grad, "dw2")):
        assert rel(got, ref) <= 5 * 2.0 ** -8, (name, rel(got, ref))


def test_swiglu_from_grouped_products_matches_expert_ffn():
    x, logits, w1, w2, _ = layer(seed=41)
    w3 = normal(44, *w1.shape, scale=w1.shape[2] ** -0.5)
    E, k, T = w1.shape[0], 4, x.shape[0]
    xg, w1g, w2g, w3g = (v.to(DEV) for v in (x, w1, w2, w3))
    ids, gates, _ = moe.route(k, logits=logits.to(DEV))
    q = moe.dispatch(ids, E, x=xg, with_x_perm=True)
    ref = moe.expert_ffn(q["offsets"], w1g, w3g, w2g, k, T, x_perm=q["x_perm"])
    # gate and up as one product with fused weights [E, 2f, d]
    gu = moe.grouped_matmul(q["x_perm"], torch.cat([w1g, w3g], 1), q["offsets"]).float()
    f = w1.shape[1]
    h = (torch.nn.functional.silu(gu[:, :f]) * gu[:, f:]).to(torch.bfloat16)
    y = moe.grouped_matmul(h, w2g, q["offsets"])
    # gate and up are rounded to bf16 here and not in the fused kernel
    # (2^-8 relative each), h and y in both
    err = torch.linalg.norm(y.double() - ref.double()) / torch.linalg.norm(ref.double())
    assert err.item() <= 5 * 2.0 ** -8


def test_int8_layer_follows_the_bf16_layer():
    """Weights quantised once, activations per token, both products in 8 bits:
    each operand's rounding is at most half a step of its row's 127, about
    amax / 254 uniform, so about amax / (254 sqrt(3)) in the mean; rows of
    normal values have amax of 3 to 4 standard deviations, hence an error of
    at most 4 / (254 sqrt(3)) = 0.92 % of each operand and sqrt(2) times that
    of a product; two products and the activation's square (which doubles a
    relative error): under 2 * 1.3 % + 1.3 %, plus the bf16 steps."""
    x, logits, w1, w2, _ = layer(seed=51)
    E, k = w1.shape[0], 4
    xg, w1g, w2g = x.to(DEV), w1.to(DEV), w2.to(DEV)
    ids, gates, _ = moe.route(k, logits=logits.to(DEV))
    q = moe.dispatch(ids, E, x=xg, with_x_perm=True)
    off = q["offsets"]
    f, d = w1.shape[1:]
    q1, s1 = moe.quantize_rows_int8(w1g.view(E * f, d))
    q2, s2 = moe.quantize_rows_int8(w2g.view(E * d, f))
    qx, sx = moe.quantize_rows_int8(q["x_perm"])
    h = moe.grouped_matmul_int8(qx, sx, q1.view(E, f, d), s1.view(E, f), off)
    qh, sh = moe.quantize_rows_int8(torch.relu(h).square())
    y8 = moe.combine(moe.grouped_matmul_int8(qh, sh, q2.view(E, d, f), s2.view(E, d), off), q["assign_pos"], gates)
    hb = torch.relu(moe.grouped_matmul(q["x_perm"], w1g, off)).square()
    yb = moe.combine(moe.grouped_matmul(hb, w2g, off), q["assign_pos"], gates)
    err = (torch.linalg.norm(y8.double() - yb.double()) / torch.linalg.norm(yb.double())).item()
    # the squared activations' rows reach 4^2 / 2 standard deviations and
    # more above their mean square: their step is up to three times as coarse
    assert err <= 0.06, err


def all_outputs(a, w, o, dc, qa, sa, qw, sw, bufs):
    moe.grouped_matmul(a, w, o, c=bufs["c"], ws=bufs["ws1"])
    moe.grouped_matmul_backward(a, w, o, dc, out=bufs["g"], ws=bufs["ws2"])
    moe.quantize_rows_int8(a, codes=qa, scales=sa)
    moe.grouped_matmul_int8(qa, sa, qw, sw, o, c=bufs["c8"], ws=bufs["ws3"])


GRAPH = [([300, 0, 77, 5], 264, 528), ([2, 1, 0, 1], 520, 2064), ([9000], 136, 144)]


def graph_state(counts, N, K, seed):
    off = offsets_of(counts)
    R, E = int(off[-1]), len(counts)
    a, w, dc = (normal(seed + i, *s).to(DEV) for i, s in enumerate([(R, K), (E, N, K), (R, N)]))
    qw, sw = moe.quantize_rows_int8(w.view(E * N, K))
    bf = torch.bfloat16
    bufs = dict(c=poisoned(R, N, dtype=bf), c8=poisoned(R, N, dtype=bf),
                g=dict(da=poisoned(R, K, dtype=bf), dw=poisoned(E, N, K, dtype=bf)),
                **{f"ws{op}": ws_for(op, R, E, N, K, bf)[0] for op in (1, 2, 3)})
    qa = torch.empty(R, K, dtype=torch.int8, device=DEV)
    sa = torch.empty(R, dtype=torch.float32, device=DEV)
    return (a, w, gpu_off(off), dc, qa, sa, qw.view(E, N, K), sw.view(E, N), bufs)


def outputs(st):
    b = st[-1]
    return dict(c=b["c"], c8=b["c8"], da=b["g"]["da"], dw=b["g"]["dw"], qa=st[4], sa=st[5])


def test_same_bits_every_time_and_in_a_replayed_graph():
    for counts, N, K in GRAPH:
        st = graph_state(counts, N, K, 60)
        all_outputs(*st)
        torch.cuda.synchronize()
        ref = {key: v.clone() for key, v in outputs(st).items()}
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            all_outputs(*st)
        torch.cuda.current_stream().wait_stream(s)
        torch.cuda.synchronize()
        for key, v in outputs(st).items():
            assert torch.equal(v, ref[key]), key
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            all_outputs(*st)
        for it in range(3):
            for v in outputs(st).values():
                v.zero_()
            for op in (1, 2, 3):
                if st[-1][f"ws{op}"] is not None:
                    st[-1][f"ws{op}"].fill_(0xFF)
            _ = (st[0].float() * 2).sum().item()
            g.replay()
            torch.cuda.synchronize()
            for key, v in outputs(st).items():
                assert torch.equal(v, ref[key]), (it, key)


def test_calls_on_two_streams_at_once():
    states = [graph_state(*GRAPH[i % len(GRAPH)], 70 + i) for i in range(4)]
    refs = []
    for st in states:
        all_outputs(*st)
        torch.cuda.synchronize()
        refs.append({key: v.clone() for key, v in outputs(st).items()})
        for v in outputs(st).values():
            v.zero_()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in states]
    for _ in range(3):
        for s, st in zip(streams, states):
            with torch.cuda.stream(s):
                all_outputs(*st)
    torch.cuda.synchronize()
    for st, ref in zip(states, refs):
        for key, v in outputs(st).items():
            assert torch.equal(v, ref[key]), key


def test_streams_of_tiles_at_once_and_replayed():
    """The largest tiles' workgroups fill the card and walk many tiles each:
    two such calls at once on two streams, and both captured and replayed
    between other work, give the bits of one call alone."""
    states = [graph_state(ragged(9000, 34, seed=s), 1272, 2048, 80 + s) for s in (1, 2)]
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


def test_more_than_2_31_elements():
    """Row offsets past 2^31 elements of c, a and dc, and past 2^32 bytes of
    w: sampled rows against the oracle."""
    R, N, K = (1 << 21) + 77, 1032, 8
    g = torch.Generator(device=DEV).manual_seed(5)
    a = torch.randn(R, K, generator=g, device=DEV).to(torch.bfloat16)
    w = torch.randn(2, N, K, generator=g, device=DEV).to(torch.bfloat16)
    off = np.array([0, 1 << 20, R], np.int32)
    c = poisoned(R, N, dtype=torch.bfloat16)
    moe.grouped_matmul(a, w, gpu_off(off), c=c)
    pick = torch.tensor([0, 1, (1 << 20) - 1, 1 << 20, R - 300, R - 1], device=DEV)
    ex = (pick >= (1 << 20)).long()
    ref = torch.einsum("rk,rnk->rn", a[pick].double().cpu(), w[ex].double().cpu()).numpy()
    terms = torch.einsum("rk,rnk->rn", a[pick].double().abs().cpu(), w[ex].double().abs().cpu()).numpy()
    check(c[pick], ref, terms, K, "bf16")
    # its gradients: dc is c
    r = moe.grouped_matmul_backward(a, w, gpu_off(off), c)
    da = torch.einsum("rn,rnk->rk", c[pick].double().cpu(), w[ex].double().cpu()).numpy()
    dat = torch.einsum("rn,rnk->rk", c[pick].double().abs().cpu(), w[ex].double().abs().cpu()).numpy()
    check(r["da"][pick], da, dat, N, "bf16")
    cols = [0, 5, N - 1]
    for e, lo, hi in G.queues(off):
        d, v = c[lo:hi][:, cols].double(), a[lo:hi].double()
        check(r["dw"][e, cols], (d.t() @ v).cpu().numpy(), (d.abs().t() @ v.abs()).cpu().numpy(), hi - lo, "bf16")
    del a, c, r
    # the last expert's weights lie beyond 2^32 bytes
    E, N, K = 130, 4096, 4104
    w = torch.empty(E, N, K, dtype=torch.bfloat16, device=DEV)
    w[-1] = torch.randn(N, K, generator=g, device=DEV)
    a = torch.randn(5, K, generator=g, device=DEV).to(torch.bfloat16)
    off = np.zeros(E + 1, np.int32)
    off[-1] = 5
    c = moe.grouped_matmul(a, w, gpu_off(off))
    ref, terms = G.matmul(f64(a), f64(w[-1:]), [0, 5])
    check(c, ref, terms, K, "bf16")
    dc = torch.randn(5, N, generator=g, device=DEV).to(torch.bfloat16)
    r = moe.grouped_matmul_backward(a, w, gpu_off(off), dc)
    (da, dat), (dw, dwt) = G.matmul_backward(f64(a), f64(w[-1:]), [0, 5], f64(dc))
    check(r["da"], da, dat, N, "bf16")
    check(r["dw"][-1:], dw, dwt, 5, "bf16")
    assert (r["dw"][:-1] == 0).all()
