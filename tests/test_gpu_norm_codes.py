"""The integer codes of qe_add_rmsnorm where the row's scale leaves the normal float32 range, or is not finite: they
are qe_quant_act's of the normed row, byte for byte, and the oracle's where its values are finite.

A scale amax / qmax below 2^-126 is rounded to a multiple of 2^-149, by up to a third of itself, so that amax over
it is not near qmax: with amax = 190 steps and 8 bits the scale is one step and the quotient 190, which is clamped.
Where the scale itself rounds to zero every code stands for zero: the library writes zeros, and the oracle, which
divides by it, is not asked.

Rows of ones have the factor 1 / sqrt(1 + 1e-6) = 1 - 5e-7, and a weight of k smallest steps times it rounds to k
steps for every k below 2^19: the normed row is the weight, exactly.
"""

import numpy as np
import pytest
import torch

from oracle import qe_oracle as O

pytestmark = pytest.mark.gpu
DEV = "cuda"
STEP = np.float32(2.0 ** -149)


@pytest.fixture(scope="module")
def L():
    from quantized_linear_moe_amd import libqe
    return libqe


def _codes(L, x, w, s, a_bits):
    """(xn, the norm's codes and scales, qe_quant_act's of xn)."""
    T, d = x.shape
    xn = torch.empty_like(x)
    own, ref = ((torch.full((T, d), 99, dtype=torch.int8, device=DEV), torch.full((T,), 99.0, device=DEV)) for _ in range(2))
    sd = None if s is None else torch.from_numpy(s).to(DEV)
    L.qe_add_rmsnorm(x, None, w, 1e-6, xn=xn, smooth=sd, a_bits=a_bits, codes=own[0], scales=own[1])
    L.qe_quant_act(xn, sd, a_bits, ref[0], ref[1])
    return xn, own, ref


@pytest.mark.parametrize("k", [1, 2, 15, 30, 31, 32, 46, 47, 62, 63, 64, 93, 127, 128, 190, 191, 254, 255, 256, 400, 8000])
@pytest.mark.parametrize("a_bits", [6, 8])
@pytest.mark.parametrize("by_factors", [False, True])
def test_subnormal_maxima(L, a_bits, k, by_factors):
    d = 72
    rng = np.random.default_rng(k)
    steps = rng.integers(-k, k + 1, d)
    steps[rng.integers(0, d, 2)] = [k, -k]
    # the values as weights, or as weights 2^89 times them and factors of 2^89
    w = np.ldexp(steps.astype(np.float32), -60 if by_factors else -149).astype(np.float32)
    s = np.full(d, 2.0 ** 89, np.float32) if by_factors else None
    x = torch.ones(3, d, device=DEV)
    x[1] = -1.0
    xn, own, ref = _codes(L, x, torch.from_numpy(w).to(DEV), s, a_bits)
    assert np.array_equal(xn[1].cpu().numpy(), -xn[0].cpu().numpy())
    if not by_factors:
        assert np.array_equal(xn[0].cpu().numpy(), steps.astype(np.float32) * STEP)
    assert torch.equal(own[0], ref[0]) and torch.equal(own[1], ref[1])
    c, sx = O.quant_act(xn.cpu().numpy(), s, a_bits)
    assert np.array_equal(own[1].cpu().numpy(), sx)
    if sx[0] > 0:
        assert np.array_equal(own[0].cpu().numpy(), c)
    else:
        assert not bool(own[0].any())


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
@pytest.mark.parametrize("a_bits", [6, 8])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_weights_that_are_not_finite(L, a_bits, dtype, bad):
    """The other channels' values and the row's scale stay qe_quant_act's (which leaves NaN out of the maximum)."""
    rng = np.random.default_rng(1)
    x = torch.from_numpy(rng.standard_normal((5, 264)).astype(np.float32)).to(dtype).to(DEV)
    w = torch.from_numpy((1 + 0.1 * rng.standard_normal(264)).astype(np.float32)).to(dtype).to(DEV)
    w[17] = bad
    w[200] = bad
    for s in (None, rng.uniform(0.5, 2.0, 264).astype(np.float32)):
        _, own, ref = _codes(L, x, w, s, a_bits)
        assert torch.equal(own[0], ref[0])
        assert torch.equal(own[1].view(torch.int32), ref[1].view(torch.int32))
