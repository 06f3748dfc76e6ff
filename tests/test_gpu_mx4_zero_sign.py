"""Microscaled code bytes with the sign of zeros: a code's sign bit is the sign of the smoothed value, also where that
is -0 or rounds to zero, whichever form of the division the neighbouring values ask for, and the norm's codes are
qe_mx4_quant's of the normed row, byte for byte.
"""

import numpy as np
import pytest
import torch

from oracle import qe_mx4_oracle as M

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module")
def L():
    from quantized_linear_moe_amd import libqe
    return libqe


def _signed(T, d, dtype, far):
    """Rows with zeros of both signs and values that round to them; far: values outside the range of the reciprocal
    form in a part of the rows."""
    rng = np.random.default_rng(T + d)
    x = rng.standard_normal((T, d)).astype(np.float32)
    x[rng.random((T, d)) < 0.2] = 0.0
    x[rng.random((T, d)) < 0.2] = -0.0
    x[rng.random((T, d)) < 0.1] *= 1e-6
    if far:
        x[::2, 7] = 1e-35
        x[::3, d - 9] = -3e34
    return torch.from_numpy(x).to(dtype)


def _quant(L, x, s, multiply=False):
    T, d = x.shape
    codes = torch.empty(T, d // 2, dtype=torch.uint8, device=DEV)
    scales = torch.empty(T, d // 32, dtype=torch.uint8, device=DEV)
    L.qe_mx4_quant(x.to(DEV), None if s is None else torch.from_numpy(s).to(DEV), codes, scales, multiply=multiply)
    return codes.cpu().numpy(), scales.cpu().numpy()


@pytest.mark.parametrize("far", [False, True])
@pytest.mark.parametrize("how", ["none", "div", "mul"])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T,d", [(1, 32), (3, 256), (64, 2048), (5, 4128)])
def test_quant_bytes(L, T, d, dtype, how, far):
    x = _signed(T, d, dtype, far)
    s = None if how == "none" else np.random.default_rng(1).uniform(0.25, 4.0, d).astype(np.float32)
    codes, scales = _quant(L, x, s, how == "mul")
    ref_c, ref_s = M.mx4_quant(M.smooth(x.float().numpy(), s, how == "mul"))
    assert np.array_equal(scales, ref_s)
    assert np.array_equal(codes, M.pack(ref_c))


@pytest.mark.parametrize("factors", ["none", "near", "far"])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T,d", [(1, 32), (9, 1536), (300, 256), (3, 18944)])
def test_norm_bytes(L, T, d, dtype, factors):
    x = _signed(T, d, dtype, False)
    rng = np.random.default_rng(2)
    w = torch.from_numpy((1 + 0.1 * rng.standard_normal(d)).astype(np.float32)).to(dtype)
    s = None if factors == "none" else rng.uniform(0.5, 2.0, d).astype(np.float32)
    if factors == "far":
        s[rng.integers(0, d, 3)] = np.float32(2.0 ** 25)
    xn = torch.empty_like(x, device=DEV)
    codes = torch.empty(T, d // 2, dtype=torch.uint8, device=DEV)
    scales = torch.empty(T, d // 32, dtype=torch.uint8, device=DEV)
    L.qe_add_rmsnorm(x.to(DEV), None, w.to(DEV), 1e-6, xn=xn, smooth=None if s is None else torch.from_numpy(s).to(DEV),
                     a_bits=4, codes=codes, scales=scales)
    assert bool((torch.signbit(xn) & (xn == 0)).any())
    own_c, own_s = _quant(L, xn, s)
    assert np.array_equal(scales.cpu().numpy(), own_s) and np.array_equal(codes.cpu().numpy(), own_c)
    ref_c, ref_s = M.mx4_quant(M.smooth(xn.float().cpu().numpy(), s, False))
    assert np.array_equal(own_s, ref_s) and np.array_equal(own_c, M.pack(ref_c))
