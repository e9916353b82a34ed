"""Pins of the 4-bit microscaled oracle: the format's values, every code's round
trip, rounding borders, the closed form of the scale, exact products."""
import numpy as np
import pytest

from oracle import moe_mxfp4 as M


def test_every_code_round_trips_at_every_scale():
    nib = np.tile(np.arange(16, dtype=np.uint8), 2)[None].repeat(255, 0)     # both halves, amax 6
    scales = M.slices(np.arange(255, dtype=np.uint8)[:, None])
    v = M.dequantize_rows(M.pack(nib), scales)
    with np.errstate(over="ignore"):
        f = v.astype(np.float32)
    # 6 * 2^(byte - 127): exact in float32 up to byte 252 (above, 6 or 4 overflow)
    ok = np.isfinite(f).all(1)
    assert ok.sum() == 253
    codes, sc = M.quantize_rows(f[ok])
    assert (codes == M.pack(nib)[ok]).all()
    assert (M.rows_of(sc, 1)[:, 0] == np.arange(255)[ok]).all()


def test_values_are_sign_exponent_and_fraction():
    for code in range(16):
        sign, e, f = code >> 3, (code >> 1) & 3, code & 1
        want = f * 0.5 if e == 0 else (1 + 0.5 * f) * 2.0 ** (e - 1)
        assert M.MAGNITUDES[code & 7] == want
        one = M.dequantize_rows(M.pack(np.full((1, 32), code)), M.slices(np.full((1, 1), 127, np.uint8)))
        assert (one == (-want if sign else want)).all()


@pytest.mark.parametrize("value,want", [
    (0.25, 0.0), (0.75, 1.0), (1.25, 1.0), (1.75, 2.0), (2.5, 2.0), (3.5, 4.0), (5.0, 4.0),
    (np.nextafter(np.float32(0.25), np.float32(1)), 0.5), (np.nextafter(np.float32(0.75), np.float32(0)), 0.5),
    (np.nextafter(np.float32(5), np.float32(9)), 6.0), (6.5, 6.0), (7.9, 6.0), (0.0, 0.0)])
def test_rounding_borders(value, want):
    x = np.full((1, 32), value, np.float32)
    x[0, 0] = 4.0    # the scale is 1
    v = M.dequantize_rows(*M.quantize_rows(np.concatenate([x, -x])))
    assert (v[0, 1:] == want).all() and (v[1, 1:] == -want).all() and v[0, 0] == 4.0


def test_scales():
    x = np.zeros((7, 32), np.float32)
    x[1, 3], x[2, 3], x[3, 3], x[4, 3] = 1.0, 7.99, 2.0 ** -140, 3.4e38
    x[5, 3], x[6, 3] = np.nan, -np.inf
    codes, s = M.quantize_rows(x)
    assert M.rows_of(s, 1)[:, 0].tolist() == [127, 125, 127, 0, 252, 255, 255]
    assert (codes[5:] == 0).all() and np.isnan(M.dequantize_rows(codes, s)[5:]).all()


def test_nearest_within_half_a_step():
    x = np.random.default_rng(0).normal(size=(64, 320)).astype(np.float32)
    codes, s = M.quantize_rows(x)
    assert s.shape == (2, 64, 8) and (s[1, :, 2:] == 127).all()
    scale = np.repeat(np.exp2(M.rows_of(s, 10).astype(np.float64) - 127), 32, 1)
    q = np.abs(x) / scale
    assert (q < 8).all() and (q.reshape(64, 10, 32).max(2) >= 4).all()
    err = np.abs(M.dequantize_rows(codes, s) - x) / scale
    half = np.where(q < 2, 0.25, np.where(q < 4, 0.5, 1.0))
    assert (err <= np.where(q > 6, q - 6, half)).all()


def test_product_is_exact_on_small_integers():
    rng = np.random.default_rng(1)
    a, w = rng.choice([-6, -4, -3, -2, -1, 0, 1, 2, 3, 4], (5, 64)), rng.choice([-2, -1, 0, 1, 2, 4], (2, 8, 64))
    a[:, ::32], w[:, :, ::32] = 4, 4
    qa, qw = M.quantize_rows(a.astype(np.float32)), M.quantize_rows(w.reshape(16, 64).astype(np.float32))
    c, _ = M.matmul(*qa, qw[0].reshape(2, 8, 32), qw[1].reshape(1, 2, 8, 8), [0, 3, 5])
    assert (c[:3] == a[:3] @ w[0].T).all() and (c[3:] == a[3:] @ w[1].T).all()
