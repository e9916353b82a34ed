"""The oracle of the grouped products pinned on the CPU: against element-wise
loops, against differences, and the quantisation against hand-computed rows."""
import numpy as np
import pytest

from oracle import moe_grouped as G
from grouped_helpers import offsets_of


def case(seed, counts, N, K, start=0, after=0):
    rng = np.random.default_rng(seed)
    off = offsets_of(counts, start)
    R = int(off[-1]) + after
    return rng.standard_normal((R, K)), rng.standard_normal((len(counts), N, K)), off, rng.standard_normal((R, N))


def test_matmul_is_its_definition():
    a, w, off, _ = case(0, [2, 0, 3], 4, 5, start=1, after=2)
    c, t = G.matmul(a, w, off)
    assert np.isnan(c[0]).all() and np.isnan(c[-2:]).all()
    for e, lo, hi in G.queues(off):
        for r in range(lo, hi):
            for n in range(4):
                assert c[r, n] == pytest.approx(sum(a[r, k] * w[e, n, k] for k in range(5)), rel=1e-13)
                assert t[r, n] == pytest.approx(sum(abs(a[r, k] * w[e, n, k]) for k in range(5)), rel=1e-13)


def test_backward_against_differences():
    a, w, off, dc = case(1, [3, 0, 4], 4, 6)
    (da, _), (dw, _) = G.matmul_backward(a, w, off, dc)
    loss = lambda a_, w_: np.sum(G.matmul(a_, w_, off)[0] * dc)  # noqa: E731
    rng = np.random.default_rng(2)
    # the loss is bilinear: a central difference has no truncation error
    for _ in range(4):
        u, v = rng.standard_normal(a.shape), rng.standard_normal(w.shape)
        assert (loss(a + u, w) - loss(a - u, w)) / 2 == pytest.approx(np.sum(da * u), rel=1e-11)
        assert (loss(a, w + v) - loss(a, w - v)) / 2 == pytest.approx(np.sum(dw * v), rel=1e-11)
    assert (dw[1] == 0).all()


def test_quantize_rows_by_hand():
    x = np.zeros((8, 16), np.float32)
    x[1, :4] = [127, -127, 0.5, 1.5]             # scale 1: ties to even
    x[2, :3] = [254, 1, -3]                      # scale 2: 0.5 -> 0, -1.5 -> -2
    x[3, 0] = np.inf
    x[4, 5] = np.nan
    x[5, :2] = [2.0 ** -149, -(2.0 ** -149)]     # subnormal: the scale's floor
    x[6, :2] = [127 * 2.0 ** -126, 2.0 ** -127]  # scale exactly 2^-126, a tie
    x[7, :2] = [np.finfo(np.float32).max, -1]
    q, s = G.quantize_rows_int8(x)
    assert s[0] == 1 and (q[0] == 0).all()
    assert s[1] == 1 and list(q[1, :4]) == [127, -127, 0, 2]
    assert s[2] == 2 and list(q[2, :3]) == [127, 0, -2]
    for r in (3, 4):
        assert np.isnan(s[r]) and (q[r] == 0).all()
    assert s[5] == np.float32(2.0 ** -126) and (q[5] == 0).all()
    assert s[6] == np.float32(2.0 ** -126) and list(q[6, :2]) == [127, 0]
    assert q[7, 0] == 127 and np.isfinite(s[7])


def test_quantize_rows_error_is_half_a_step():
    rng = np.random.default_rng(3)
    x = (rng.standard_normal((50, 64)) * np.exp(4 * rng.standard_normal((50, 1)))).astype(np.float32)
    q, s = G.quantize_rows_int8(x)
    assert (np.abs(q.astype(np.int32)).max(1) == 127).all()
    err = np.abs(q.astype(np.float64) * s[:, None].astype(np.float64) - x)
    # half a step, and the quotient's own rounding (2^-24 of at most 127 steps)
    assert (err <= s[:, None].astype(np.float64) * (0.5 + 127 * 2.0 ** -23)).all()


def test_int8_product_is_its_definition():
    rng = np.random.default_rng(4)
    off = offsets_of([2, 0, 1])
    qa = rng.integers(-127, 128, (3, 16)).astype(np.int8)
    qw = rng.integers(-128, 128, (3, 5, 16)).astype(np.int8)
    sa, sw = rng.random(3).astype(np.float32), rng.random((3, 5)).astype(np.float32)
    c = G.matmul_int8(qa, sa, qw, sw, off)
    for e, lo, hi in G.queues(off):
        for r in range(lo, hi):
            for n in range(5):
                t = sum(int(qa[r, k]) * int(qw[e, n, k]) for k in range(16))
                assert c[r, n] == pytest.approx(t * float(sa[r]) * float(sw[e, n]), rel=1e-14)
