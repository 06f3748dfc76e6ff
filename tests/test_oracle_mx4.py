"""Pins of the microscaled 4-bit oracle and of the norm oracle: values worked by hand, and properties."""

import numpy as np

from oracle import qe_mx4_oracle as M


def _block(*values):
    x = np.zeros((1, 32), np.float32)
    x[0, : len(values)] = values
    return x


def test_hand_worked_block():
    # amax 7 in [4, 8): E = 2, scale 1 (byte 127); 7 saturates to 6
    codes, scales = M.mx4_quant(_block(7.0, -0.25, 0.25001, 0.75, 1.25, -1.75, 2.5, 3.5, 5.0, 5.0001, -0.0))
    assert scales[0, 0] == 127
    # ties go to the even index: 0.25 -> 0, 0.75 -> 1 (index 2), 1.25 -> 1, 1.75 -> 2, 2.5 -> 2, 3.5 -> 4, 5 -> 4
    assert codes[0, :11].tolist() == [7, 8 + 0, 1, 2, 2, 8 + 4, 4, 6, 6, 7, 8]


def test_scale_of_powers_of_two_and_limits():
    for amax, byte in ((1.0, 125), (0.999, 124), (1.999, 125), (2.0, 126), (6.0, 127), (8.0, 128),
                       (3.4028235e38, 252), (2.0 ** -124, 1), (2.0 ** -125, 0), (2.0 ** -126, 0), (1e-45, 0), (0.0, 0)):
        codes, scales = M.mx4_quant(_block(amax))
        assert scales[0, 0] == byte, amax
    # the largest magnitude lands in [4, 8) scales, so it is 4 or 6 of them
    assert M.mx4_quant(_block(1.0))[0][0, 0] == 6 and M.mx4_quant(_block(1.999))[0][0, 0] == 7


def test_non_finite_blocks_are_nan():
    for bad in (np.nan, np.inf, -np.inf):
        x = np.concatenate([_block(1.0, bad), _block(1.0, 2.0)], axis=1)
        codes, scales = M.mx4_quant(x)
        assert scales.tolist() == [[255, 126]] and not codes[0, :32].any()
        v = M.mx4_values(codes, scales)
        assert np.isnan(v[0, :32]).all() and v[0, 32] == 1.0 and v[0, 33] == 2.0


def test_values_round_trip_and_error_bound():
    rng = np.random.default_rng(0)
    x = (rng.standard_normal((64, 96)) * np.exp2(rng.integers(-20, 20, (64, 1)))).astype(np.float32)
    codes, scales = M.mx4_quant(x)
    v = M.mx4_values(codes, scales)
    again = M.mx4_quant(v.astype(np.float32))
    # a block whose largest magnitude saturated keeps its scale too (6 scales is in [4, 8))
    assert np.array_equal(again[0] & 7, codes & 7) and np.array_equal(again[1], scales)
    s = np.repeat(np.ldexp(1.0, scales.astype(int) - 127), 32, axis=1)
    # half a spacing below 6 scales (at most 1 scale), and up to 2 scales where a value saturates
    err = np.abs(v - x) / s
    assert np.all(err[np.abs(x) <= 6 * s] <= 1.0) and np.all(err < 2.0)
    assert np.array_equal(M.unpack(M.pack(codes)), codes)


def test_norm_hand_worked():
    # h = (3, 4, 0, ..., 0) over 8 channels: mean square 25/8
    x = np.zeros((1, 8), np.float32)
    x[0, 0], x[0, 1] = 1.0, 4.0
    r = np.zeros((1, 8), np.float32)
    r[0, 0] = 2.0
    h, xn = M.add_rmsnorm(x, r, np.full(8, 2.0, np.float32), 1e-20, False)
    f = np.float32(1.0 / np.sqrt(25.0 / 8.0))
    assert h[0, :2].tolist() == [3.0, 4.0]
    assert xn[0, 0] == np.float32(3.0) * f * np.float32(2.0) and xn[0, 1] == np.float32(4.0) * f * np.float32(2.0)
    assert not xn[0, 2:].any()
    # rows of unit mean square come out as the weight times the row
    x = np.where(np.arange(64) % 2, 1.0, -1.0).astype(np.float32)[None, :]
    _, xn = M.add_rmsnorm(x, None, np.arange(64, dtype=np.float32), 1e-30, False)
    assert np.array_equal(xn[0], x[0] * np.arange(64))


def test_gemm_sums_terms():
    rng = np.random.default_rng(1)
    a, w = rng.integers(-3, 4, (5, 64)).astype(float), rng.integers(-3, 4, (6, 64)).astype(float)
    u, B_s = rng.integers(-2, 3, (5, 3)), rng.integers(-2, 3, (3, 6))
    v, B_r, e = rng.integers(-2, 3, (5, 2)), rng.integers(-2, 3, (4, 2, 6)), np.array([0, 3, 3, 1, 2])
    y, mag = M.mx4_gemm(a, w, u, B_s, v, e, B_r)
    for t in range(5):
        for i in range(6):
            want = sum(a[t, j] * w[i, j] for j in range(64)) + sum(u[t, k] * B_s[k, i] for k in range(3)) + \
                sum(v[t, k] * B_r[e[t], k, i] for k in range(2))
            assert y[t, i] == want and mag[t, i] >= abs(want)
