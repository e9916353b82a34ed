"""4-bit microscaled floats on the GPU: codes and scales bit for bit against the
oracle (``oracle.moe_mxfp4``), their numbers exactly, products within the bound
of a float32 accumulation (``grouped_helpers.check``)."""
import numpy as np
import pytest
import torch

import mixture_experts_layer_exclusive_amd as moe
from grouped_helpers import DEV, QUEUES, TORCH, check, f64, normal, offsets_of
from oracle import moe_mxfp4 as M

pytestmark = pytest.mark.gpu

WIDTHS = [(8, 32), (64, 256), (72, 96), (136, 288), (256, 1056), (520, 64), (1000, 544)]
LARGE = {
    "ragged": ([1900, 0, 1, 2500, 300, 3491], 2056, 544),
    "one queue": ([4100], 4104, 224),
    # more tiles of 256 than twice the CUs, of several slices, the last not whole: over
    # and under 8 columns of tiles
    "stream": ([2900, 1, 0, 2555, 3556], 4360, 800),
    "stream of few columns": ([20001, 300, 19000], 1032, 544),
}
# (kernel, rows, E, N, K)
CHOICES = [("split32", 11, 3, 1440, 480), ("split32", 327, 17, 16, 608), ("split64", 231, 1, 2744, 3296),
           ("split64", 225, 1, 2680, 3488), ("tile64x128", 1801, 2, 640, 992), ("tile64x128", 1263, 2, 552, 1248),
           ("tile64x128", 1500, 17, 1680, 96), ("short", 33, 17, 1680, 96), ("short", 300, 5, 520, 160),
           ("short", 900, 17, 1160, 256), ("short", 130, 200, 1000, 224), ("short", 64, 1, 2056, 64),
           ("tile128", 620, 1, 4600, 1056), ("tile128", 4079, 17, 440, 800), ("tile128", 375, 1, 7744, 1120),
           ("tile256", 5180, 5, 1560, 2560), ("tile256", 2131, 1, 4024, 2496),
           ("tile128x256", 999, 8, 3400, 1600), ("tile128x256", 1875, 3, 2168, 1568),
           ("tile128x256", 3662, 1, 1064, 2656), ("halves64x128", 756, 3, 1184, 3936),
           ("halves64x128", 264, 5, 2256, 3392), ("halves64x128", 480, 1, 2320, 8704),
           ("halves64x128", 818, 3, 1552, 4608), ("halves128", 1175, 3, 1832, 4704),
           ("halves128", 820, 1, 2584, 5120), ("halves128", 642, 1, 3096, 5728)]
DENSE = [(1, 8, 32), (1, 4096, 2048), (16, 1000, 8224), (33, 136, 131104), (300, 520, 4096), (4100, 2056, 544)]


def gpu(a):
    return torch.from_numpy(np.ascontiguousarray(a)).to(DEV)


def quantised(seed, *shape, spread=2.0):
    """Random codes (every one of them) and scale bytes around 127."""
    rng = np.random.default_rng(seed)
    *rows, cols = shape
    n = int(np.prod(rows))
    codes = rng.integers(0, 256, (n, cols // 2), dtype=np.uint8)
    bytes_ = np.clip(np.rint(127 + spread * rng.normal(size=(n, cols // 32))), 0, 254).astype(np.uint8)
    return codes, M.slices(bytes_)


# ---- quantise --------------------------------------------------------------------

def check_quantise(x):
    """x: a CPU tensor [rows, cols]."""
    rows, cols = x.shape
    codes = torch.full((rows, cols // 2), 0xEE, dtype=torch.uint8, device=DEV)
    scales = torch.full((-(-cols // 256), rows, 8), 0xEE, dtype=torch.uint8, device=DEV)
    moe.quantize_rows_mxfp4(x.to(DEV), codes=codes, scales=scales)
    torch.cuda.synchronize()
    want, sw = M.quantize_rows(x.float().numpy())
    assert (scales.cpu().numpy() == sw).all()
    got = codes.cpu().numpy()
    assert (got == want).all(), (np.argwhere(got != want)[:3], got[got != want][:3], want[got != want][:3])
    ref = M.dequantize_rows(want, sw)
    for dtype in (torch.float32, torch.bfloat16):
        v = moe.dequantize_rows_mxfp4(codes, scales, dtype=dtype)
        np.testing.assert_array_equal(f64(v), np.where(np.abs(ref) >= 2.0 ** 128, np.copysign(np.inf, ref), ref))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,cols", [(1, 32), (3, 64), (7, 224), (5, 256), (33, 288), (129, 1056), (16, 4096), (1, 65536),
                                       (2000, 96), (2, 20512)])
def test_quantise(rows, cols, dtype):
    x = normal(rows + cols, rows, cols) * torch.exp(2 * normal(1, rows, 1).float()).to(torch.bfloat16)
    check_quantise(x.to(TORCH[dtype]) if dtype == "bf16" else normal(rows, rows, cols, dtype="f32") * x.float())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,cols", [(4099, 2080), (8192, 1024), (131, 65504)])
def test_quantise_large(rows, cols, dtype):
    """Enough for a slice of rows per workgroup; rows and columns that end inside one."""
    x = normal(rows, rows, cols, dtype=dtype)
    x[rows - 1, cols - 5], x[7, 300] = np.nan, np.inf
    x[11, 320:352] = 0
    check_quantise(x)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_quantise_borders(dtype):
    """Every rounding border and its neighbours, at every scale of the type."""
    base = np.array([0, 0.25, 0.5, 0.75, 1, 1.25, 1.5, 1.75, 2, 2.5, 3, 3.5, 4, 5, 6, 7], np.float32)
    t = torch.from_numpy(base).to(TORCH[dtype])
    around = [t]
    ints = torch.int16 if dtype == "bf16" else torch.int32
    for step in (-1, 1):
        around.append((t[1:].view(ints) + step).view(TORCH[dtype]))
    v = torch.cat(around + [-a for a in around])
    blocks = []
    for i in range(0, v.numel(), 31):
        b = torch.full((32,), 4.0, dtype=TORCH[dtype])
        part = v[i:i + 31]
        b[1:1 + part.numel()] = part
        blocks.append(b)
    x = torch.cat(blocks)
    rows = torch.stack([(x.double() * 2.0 ** e).to(TORCH[dtype]) for e in range(-150, 126, 3)])
    check_quantise(rows)


def test_quantise_special_blocks():
    x = normal(0, 8, 320, dtype="f32")
    x[0, 3], x[1, 40], x[2, 100], x[2, 101] = np.nan, np.inf, -np.inf, np.nan
    x[3] = 0
    x[4] = -0.0
    x[5] = torch.finfo(torch.float32).max
    x[6] = 2.0 ** -149
    x[7, :32] = torch.finfo(torch.float32).min
    check_quantise(x)
    check_quantise(x.to(torch.bfloat16))


def test_dequantise_every_byte():
    nib = np.tile(np.arange(16, dtype=np.uint8), (256, 2))
    codes, scales = M.pack(nib), M.slices(np.arange(256, dtype=np.uint8)[:, None])
    ref = M.dequantize_rows(codes, scales)
    ref = np.where(np.abs(ref) >= 2.0 ** 128, np.copysign(np.inf, ref), ref)
    for dtype in (torch.float32, torch.bfloat16):
        np.testing.assert_array_equal(f64(moe.dequantize_rows_mxfp4(gpu(codes), gpu(scales), dtype=dtype)), ref)


def test_no_rows():
    c, s = moe.quantize_rows_mxfp4(torch.empty(0, 64, dtype=torch.bfloat16, device=DEV))
    assert c.shape == (0, 32) and s.shape == (1, 0, 8)
    assert moe.dequantize_rows_mxfp4(c, s).shape == (0, 64)
    out = moe.grouped_matmul_mxfp4(c, s, torch.zeros(2, 8, 32, dtype=torch.uint8, device=DEV),
                                   torch.zeros(1, 2, 8, 8, dtype=torch.uint8, device=DEV), gpu(np.zeros(3, np.int32)))
    assert out.shape == (0, 8)


# ---- product -----------------------------------------------------------------------

def product(a, w, off, N, dtype, E=None, what=""):
    """a, w: (codes, scales); off None: dense."""
    R, K = a[0].shape[0], 2 * a[0].shape[1]
    dense = off is None
    E = 1 if dense else len(off) - 1
    wc, ws = w[0].reshape(E, N, K // 2), w[1].reshape(-1, E, N, 8)
    c = torch.full((R, N), 3.0e4, dtype=TORCH[dtype], device=DEV)
    moe.grouped_matmul_mxfp4(gpu(a[0]), gpu(a[1]), gpu(wc[0] if dense else wc), gpu(ws[:, 0] if dense else ws),
                             None if dense else gpu(off), out_dtype=TORCH[dtype], c=c)
    torch.cuda.synchronize()
    ref, terms = M.matmul(*a, wc, ws, [0, R] if dense else off)
    check(c, ref, terms, K, dtype, what)
    outside = np.isnan(ref) & ~np.isnan(terms)
    assert (f64(c)[outside] == f64(torch.tensor(3.0e4, dtype=TORCH[dtype]))).all(), "a row outside the queues was written"
    return c


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("N,K", WIDTHS)
@pytest.mark.parametrize("queues", list(QUEUES))
def test_product(queues, N, K, dtype):
    counts = QUEUES[queues]
    if len(counts) * N * K > 4e7:
        N, K = min(N, 136), min(K, 288)
    off = offsets_of(counts, start=3)
    R = int(off[-1]) + 5
    product(quantised(1, R, K), quantised(2, len(counts), N, K), off, N, dtype, what=f"{queues} {N}x{K}")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("queues", list(LARGE))
def test_product_large(queues, dtype):
    counts, N, K = LARGE[queues]
    off = offsets_of(counts, start=2)
    R = int(off[-1]) + 8
    product(quantised(3, R, K), quantised(4, len(counts), N, K), off, N, dtype, what=queues)


def ragged(rows, E, seed):
    w = np.random.default_rng(seed).random(E) ** 2
    c = np.floor(rows * w / w.sum()).astype(int)
    c[0] += rows - c.sum()
    return c.tolist()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("kernel,rows,E,N,K", CHOICES)
def test_every_kernel(kernel, rows, E, N, K, dtype):
    off = offsets_of(ragged(rows - 7, E, seed=rows), start=3)
    product(quantised(20, rows, K), quantised(21, E, N, K), off, N, dtype, what=kernel)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,N,K", DENSE)
def test_dense(rows, N, K, dtype):
    product(quantised(5, rows, K), quantised(6, N, K), None, N, dtype, what=f"dense {rows} {N}x{K}")


def test_scales_of_blocks_past_the_row_do_not_matter():
    off = offsets_of([40, 0, 90])
    for N, K in ((72, 96), (264, 1056), (136, 32)):
        a, w = quantised(7, 130, K), quantised(8, 3, N, K)
        c = product(a, w, off, N, "f32")
        blocks = K // 32 % 8
        for s in (a[1], w[1]):
            s[-1, :, blocks:] = np.random.default_rng(0).choice([0, 1, 254, 255], s[-1, :, blocks:].shape)
        d = product(a, w, off, N, "f32")
        assert torch.equal(c, d)


def test_scales_over_their_whole_range():
    """Exponents from -127 to 127 in both operands, in pairs whose products stay
    finite: float32 results from 2^-126 (below: see the bound) to 2^126."""
    rng = np.random.default_rng(9)
    R, N, K = 64, 64, 512
    a, w = quantised(10, R, K), quantised(11, 1, N, K)
    for e in (-120, -60, 0, 60, 110):
        # a row of one exponent, columns of the opposite one
        row = np.clip(127 + e + rng.integers(-3, 4, (R, K // 32)), 0, 254).astype(np.uint8)
        col = np.clip(127 - e + rng.integers(-3, 4, (N, K // 32)), 0, 254).astype(np.uint8)
        product((a[0], M.slices(row)), (w[0], M.slices(col)), offsets_of([R]), N, "f32", what=str(e))


def test_nan_blocks():
    """A block of scale 255 makes its row, or its column, NaN, and no other."""
    for R, N, K in ((70, 72, 96), (300, 264, 1056), (33, 520, 288)):
        a, w = quantised(12, R, K), quantised(13, 1, N, K)
        a[0][5], w[0][9] = 0, 0        # (also where the codes are zero)
        a[1][0, 5, 1] = 255
        w[1][-1, 9, 0] = 255
        c = torch.full((R, N), 3.0e4, dtype=torch.float32, device=DEV)
        moe.grouped_matmul_mxfp4(gpu(a[0]), gpu(a[1]), gpu(w[0][None] if w[0].ndim == 2 else w[0]), gpu(w[1][:, None]),
                                 gpu(offsets_of([R])), out_dtype=torch.float32, c=c)
        got = np.isnan(f64(c))
        want = np.zeros((R, N), bool)
        want[5], want[:, 9] = True, True
        assert (got == want).all()


@pytest.mark.parametrize("counts", [[2, 3], [70, 3], [300, 20], [1000, 600]])
def test_nan_behind_a_queue_stays_there(counts):
    """Rows of the next queue, and columns of the next expert, lie in a tile's
    reach: their NaN does not enter."""
    N, K = 72, 96
    off = offsets_of(counts)
    R = int(off[-1])
    a, w = quantised(14, R, K), quantised(15, 2, N, K)
    a[1][:, counts[0]:] = 255
    w[1].reshape(-1, 2, N, 8)[:, 1] = 255
    c = moe.grouped_matmul_mxfp4(gpu(a[0]), gpu(a[1]), gpu(w[0].reshape(2, N, -1)), gpu(w[1].reshape(-1, 2, N, 8)), gpu(off))
    got = np.isnan(f64(c))
    assert not got[:counts[0]].any() and got[counts[0]:].all()


def test_broken_offsets_stay_inside():
    R, N, K, E = 200, 72, 96, 4
    a, w = quantised(16, R, K), quantised(17, E, N, K)
    guard = torch.full((3, R, N), 3.0e4, dtype=torch.bfloat16, device=DEV)
    for off in ([-5, 60, 20, 300, 900], [2 ** 31 - 1] * 5, [-2 ** 31, 2 ** 31 - 1, -1, 5, 7], [0, 0, 0, 0, 2 ** 30]):
        moe.grouped_matmul_mxfp4(gpu(a[0]), gpu(a[1]), gpu(w[0].reshape(E, N, -1)), gpu(w[1].reshape(-1, E, N, 8)),
                                 gpu(np.array(off, np.int32)), c=guard[1])
        torch.cuda.synchronize()
        assert (guard[0] == 3.0e4).all() and (guard[2] == 3.0e4).all()


@pytest.mark.parametrize("kernel,rows,E,N,K", [c for c in CHOICES if c[2] >= 3])
def test_nan_and_broken_offsets_at_every_kernel(kernel, rows, E, N, K):
    """As above, at the sizes of every kernel with queues: expert 1's rows and weights are
    NaN; then offsets that are no offsets, with guards on both sides."""
    counts = ragged(rows, E, seed=1)
    off = offsets_of(counts)
    a, w = quantised(21, rows, K), quantised(22, E, N, K)
    ac, wc, dense = gpu(a[0]), gpu(w[0].reshape(E, N, -1)), gpu(w[1].reshape(-1, E, N, 8))
    nan_a, nan_w = gpu(a[1]), dense.clone()
    nan_a[:, off[1]:off[2]] = 255
    nan_w[:, 1] = 255
    c = moe.grouped_matmul_mxfp4(ac, nan_a, wc, nan_w, gpu(off))
    clean = moe.grouped_matmul_mxfp4(ac, gpu(a[1]), wc, dense, gpu(off))
    assert torch.isnan(c[off[1]:off[2]]).all()
    for lo, hi in ((off[0], off[1]), (off[2], off[E])):
        assert torch.equal(c[lo:hi], clean[lo:hi]) and not torch.isnan(c[lo:hi]).any()
    guard = torch.full((3, rows, N), 3.0e4, dtype=torch.bfloat16, device=DEV)
    for bad in ([-5] + [rows // 2, 20] * E, [2 ** 31 - 1] * (E + 1), [0] * E + [2 ** 30]):
        moe.grouped_matmul_mxfp4(ac, gpu(a[1]), wc, dense, gpu(np.array(bad[:E + 1], np.int32)), c=guard[1])
        torch.cuda.synchronize()
        assert (guard[0] == 3.0e4).all() and (guard[2] == 3.0e4).all()


def test_same_bits_again_and_captured():
    counts, N, K = [700, 1, 0, 2, 320], 520, 1056
    off, R = gpu(offsets_of(counts)), sum(counts)
    x = normal(18, R, K).to(DEV)
    w = moe.quantize_rows_mxfp4(normal(19, 5 * N, K).to(DEV))
    wc, ws = w[0].view(5, N, -1), w[1].view(-1, 5, N, 8)

    def step():
        a, s = moe.quantize_rows_mxfp4(x)
        return moe.grouped_matmul_mxfp4(a, s, wc, ws, off), moe.dequantize_rows_mxfp4(a, s)

    first = step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step()
    for seed in range(4):
        if seed:
            x.copy_(normal(30 + seed, R, K))
        graph.replay()
        torch.cuda.synchronize()
        got = [h.clone() for h in held]
        want = step() if seed else first
        assert all(torch.equal(a, b) for a, b in zip(got, want))


# ---- the operators together, as a layer uses them ----------------------------------

def test_layer_of_parts_trains():
    """Scored routing -> dispatch -> 4-bit products around a squared ReLU ->
    combine, and back: straight through the quantisation, on the dequantised
    weights.  Every gradient against torch's automatic differentiation in 64 bits
    of the same layer over the same codes."""
    T, d, f, E, k, scale = 200, 128, 160, 16, 4, 2.0
    g = torch.Generator().manual_seed(3)
    rand = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    x = rand(T, d).to(DEV).bfloat16()
    wr = (0.2 * rand(E, d)).to(DEV).bfloat16()
    w1, w2 = (rand(E, f, d) / d ** 0.5).to(DEV).bfloat16(), (rand(E, d, f) / f ** 0.5).to(DEV).bfloat16()
    bias, dy = (0.05 * rand(E)).to(DEV), rand(T, d).to(DEV).bfloat16()
    balance = (rand(E) / T).to(DEV)
    cfg = dict(score="sigmoid", scale=scale)

    ids, gates, logits, sums = moe.route_scored(k, x=x, w_router=wr, bias=bias, groups=4, groups_kept=2,
                                                with_score_sums=True, **cfg)
    q = moe.dispatch(ids, E, x=x, with_x_perm=True)
    q1, q2 = moe.quantize_rows_mxfp4(w1.view(E * f, d)), moe.quantize_rows_mxfp4(w2.view(E * d, f))
    xa = moe.quantize_rows_mxfp4(q["x_perm"])
    u = moe.grouped_matmul_mxfp4(*xa, q1[0].view(E, f, -1), q1[1].view(-1, E, f, 8), q["offsets"])
    h = torch.relu(u).square()
    ha = moe.quantize_rows_mxfp4(h)
    y_perm = moe.grouped_matmul_mxfp4(*ha, q2[0].view(E, d, -1), q2[1].view(-1, E, d, 8), q["offsets"])
    y = moe.combine(y_perm, q["assign_pos"], gates)

    v1, v2 = moe.dequantize_rows_mxfp4(*q1).view(E, f, d), moe.dequantize_rows_mxfp4(*q2).view(E, d, f)
    xv, hv = moe.dequantize_rows_mxfp4(*xa), moe.dequantize_rows_mxfp4(*ha)
    c = moe.combine_backward(dy, q["assign_pos"], gates, y_perm=y_perm)
    g2 = moe.grouped_matmul_backward(hv, v2, q["offsets"], c["dy_perm"])
    du = (g2["da"] * 2 * torch.relu(u)).to(torch.bfloat16)
    g1 = moe.grouped_matmul_backward(xv, v1, q["offsets"], du)
    dl = moe.route_scored_backward(logits, ids, c["dgates"], dscore_sums=balance, dtype=torch.bfloat16, **cfg)
    all_rows = torch.tensor([0, T], dtype=torch.int32, device=DEV)
    gr = moe.grouped_matmul_backward(x, wr[None], all_rows, dl)
    ones = torch.ones(T, k, device=DEV)
    dx = moe.combine(g1["da"], q["assign_pos"], ones).double() + gr["da"].double()
    torch.cuda.synchronize()

    # 64 bits on the CPU, the quantised values standing in, gradients passing them
    D = lambda t: t.detach().double().cpu()  # noqa: E731
    X, WR, V1, V2 = (D(t).requires_grad_(True) for t in (x, wr, v1, v2))
    s = torch.sigmoid(X @ WR.t())
    I = ids.cpu().long()
    G = s.gather(1, I)
    G = scale * G / G.sum(1, keepdim=True)
    pos = q["assign_pos"].cpu().long().view(T, k)
    token = torch.empty(T * k, dtype=torch.long)
    token[pos.view(-1)] = torch.arange(T * k) // k
    expert = torch.empty(T * k, dtype=torch.long)
    expert[pos.view(-1)] = I.reshape(-1)
    XP = X[token]
    XP = XP + (D(xv) - XP).detach()
    U1 = torch.stack([V1[e] @ XP[r] for r, e in enumerate(expert.tolist())])
    H = torch.relu(U1).square()
    H = H + (D(hv) - H).detach()
    YP = torch.stack([V2[e] @ H[r] for r, e in enumerate(expert.tolist())])
    Y = (G[:, :, None] * YP[pos]).sum(1)
    loss = (Y * D(dy)).sum() + (s.sum(0) * D(balance)).sum()
    want = torch.autograd.grad(loss, (X, WR, V1, V2))

    def off(got, ref):
        return ((D(got) - ref.detach()).norm() / ref.detach().norm()).item()

    # bf16 values in between (u, y_perm, dy_perm, da, du, dl, and the results): each
    # rounds by at most 2^-8 of a value, so any of these sums is off by at most 8 of
    # them relative to the sum of its terms' norms; norms of sums of terms of random
    # sign and of their roundings shrink alike
    assert off(y, Y) < 8 * 2.0 ** -8 and off(sums, s.sum(0)) < 1e-5
    for got, ref, name in zip((dx, gr["dw"][0], g1["dw"], g2["dw"]), want, ("dx", "dw_router", "dw1", "dw2")):
        assert off(got, ref) < 8 * 2.0 ** -8, (name, off(got, ref))
