"""Oracle of the microscaled 4-bit operators and of the residual addition with RMS norm (numpy, float64).

Written from the definitions (OCP Microscaling Formats specification, version 1.0: MXFP4 is blocks of
32 elements of type E2M1 with an E8M0 scale), sharing no code with the library.  Test infrastructure.
"""

import numpy as np

from . import qe_oracle as O

LEVELS = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def mx4_quant(x: np.ndarray):
    """(codes uint8 [T, d], scale bytes uint8 [T, d/32]) of float32 x, one code per entry."""
    x = np.asarray(x, dtype=np.float32)
    T, d = x.shape
    b = x.astype(np.float64).reshape(T, d // 32, 32)
    mag = np.abs(b)
    bad = ~np.isfinite(mag).all(axis=-1)
    amax = np.where(bad, 0.0, np.where(np.isfinite(mag), mag, 0.0).max(axis=-1))
    _, e = np.frexp(amax)  # amax = m 2^e with m in [1/2, 1): floor(log2 amax) = e - 1
    byte = np.where(amax > 0, np.maximum(e - 1 - 2 + 127, 0), 0)
    r = np.where(np.isfinite(mag), mag, 0.0) / np.ldexp(1.0, byte - 127)[..., None]
    # nearest level; of two at the same distance the one with the even index
    dist = np.abs(r[..., None] - LEVELS)
    code = np.argmin(dist, axis=-1)
    up = np.minimum(code + 1, 7)
    tie = (np.take_along_axis(dist, up[..., None], -1)[..., 0] == dist.min(axis=-1)) & (up != code)
    code = np.where(tie & (code % 2 == 1), up, code)
    code = code + 8 * np.signbit(b)
    code = np.where(bad[..., None], 0, code)
    byte = np.where(bad, 255, byte)
    return code.reshape(T, d).astype(np.uint8), byte.astype(np.uint8)


def pack(codes: np.ndarray) -> np.ndarray:
    """[T, d] codes to [T, d/2] bytes, even channels in the low nibble."""
    return (codes[:, 0::2] | (codes[:, 1::2] << 4)).astype(np.uint8)


def unpack(packed: np.ndarray) -> np.ndarray:
    out = np.empty((packed.shape[0], packed.shape[1] * 2), np.uint8)
    out[:, 0::2] = packed & 15
    out[:, 1::2] = packed >> 4
    return out


def mx4_values(codes: np.ndarray, scales: np.ndarray) -> np.ndarray:
    """float64 values of [T, d] codes and [T, d/32] scale bytes."""
    v = LEVELS[codes & 7] * np.where(codes & 8, -1.0, 1.0)
    s = np.where(scales == 255, np.nan, np.ldexp(1.0, scales.astype(np.int64) - 127))
    return v * np.repeat(s, 32, axis=1)


def smooth(x: np.ndarray, s, multiply: bool) -> np.ndarray:
    x = np.asarray(x, dtype=np.float32)
    if s is None:
        return x
    s = np.asarray(s, dtype=np.float32)
    return x * s if multiply else x / s


def mx4_gemm(a: np.ndarray, w: np.ndarray, u=None, B_s=None, v=None, expert=None, B_r=None):
    """float64 y and the sum of the terms' magnitudes (for error bounds).  a, w: values."""
    y, mag = a @ w.T, np.abs(a) @ np.abs(w).T
    if u is not None:
        u, B = np.asarray(u, np.float64), np.asarray(B_s, np.float64)
        y, mag = y + u @ B, mag + np.abs(u) @ np.abs(B)
    if v is not None:
        v, B = np.asarray(v, np.float64), np.asarray(B_r, np.float64)
        y, mag = y.copy(), mag.copy()
        for e in range(B.shape[0]):
            at = np.nonzero(expert == e)[0]
            y[at] += v[at] @ B[e]
            mag[at] += np.abs(v[at]) @ np.abs(B[e])
    return y, mag


def add_rmsnorm(x, res, weight, eps: float, bf16: bool):
    """(h, xn) float32 holding values of the row's type: the sum of squares, its root and the quotient
    in float64, the factor rounded to float32, the two products in float32, one rounding at the end."""
    rn = (lambda t: O.bf16_round(t)) if bf16 else (lambda t: t.astype(np.float32))
    x = np.asarray(x, np.float32)
    h = x if res is None else rn(x + np.asarray(res, np.float32))
    m = np.sum(h.astype(np.float64) ** 2, axis=1, keepdims=True) / x.shape[1]
    r = (1.0 / np.sqrt(m + np.float64(np.float32(eps)))).astype(np.float32)
    return h, rn((h * r) * np.asarray(weight, np.float32)[None, :])
