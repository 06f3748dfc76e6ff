"""GPU parity of the residual addition with RMS norm and of its quantized outputs.

h is one float32 addition and one rounding; the norm's factor comes from a float64 sum rounded to
float32, whose last place the order of the additions does not reach (a float64 sum of at most 32768 squares is
off by less than 2^-37 relative, and a factor that close to a rounding border does not occur in these fixed
inputs); the two products are float32 operations.  So h, xn and the codes are compared bit for bit: xn
with the oracle, the codes with the oracle's codes of xn and with the library's own quantization of xn.
"""

import numpy as np
import pytest
import torch

from oracle import qe_mx4_oracle as M
from oracle import qe_oracle as O

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module")
def L():
    from quantized_linear_moe_amd import libqe
    return libqe


def _inputs(T, d, dtype, seed=0):
    rng = np.random.default_rng(seed + T * 7 + d)
    x = rng.standard_normal((T, d)).astype(np.float32)
    x[:, rng.integers(0, d, 2)] *= 30.0
    r = rng.standard_normal((T, d)).astype(np.float32)
    w = (1 + 0.1 * rng.standard_normal(d)).astype(np.float32)
    s = rng.uniform(0.5, 2.0, d).astype(np.float32)
    t = lambda a: torch.from_numpy(a).to(dtype)  # noqa: E731
    return t(x), t(r), t(w), s


def _codes_for(T, d, a_bits):
    if a_bits == 4:
        return (torch.full((T + 1, d // 2), 77, dtype=torch.uint8, device=DEV),
                torch.full((T + 1, d // 32), 77, dtype=torch.uint8, device=DEV))
    return (torch.full((T + 1, d), 77, dtype=torch.int8, device=DEV),
            torch.full((T + 1,), 77.0, dtype=torch.float32, device=DEV))


def _run(L, x, res, w, s, a_bits, eps=1e-6, want_h=True, want_xn=True):
    """The call on outputs with one sentinel row behind the last; returns (h, xn, codes, scales)."""
    T, d = x.shape
    big = lambda: torch.full((T + 1, d), 77.0, dtype=x.dtype, device=DEV)  # noqa: E731
    h, xn = big() if want_h else None, big() if want_xn else None
    codes, scales = _codes_for(T, d, a_bits) if a_bits else (None, None)
    cut = lambda t: None if t is None else t[:T]  # noqa: E731
    L.qe_add_rmsnorm(x.to(DEV), None if res is None else res.to(DEV), w.to(DEV), eps, h=cut(h), xn=cut(xn),
                     smooth=None if s is None else torch.from_numpy(s).to(DEV), a_bits=a_bits, codes=cut(codes),
                     scales=cut(scales))
    torch.cuda.synchronize()
    for t in (h, xn, codes, scales):
        if t is not None:
            assert bool((t[T:] == 77).all()), "the row behind the last was written"
    return cut(h), cut(xn), cut(codes), cut(scales)


def _check(L, x, res, w, s, a_bits, got, eps=1e-6):
    h, xn, codes, scales = got
    bf = x.dtype == torch.bfloat16
    ref_h, ref_xn = M.add_rmsnorm(x.float().numpy(), None if res is None else res.float().numpy(), w.float().numpy(), eps, bf)
    if h is not None:
        assert np.array_equal(h.float().cpu().numpy(), ref_h)
    if xn is not None:
        assert np.array_equal(xn.float().cpu().numpy(), ref_xn)
    if a_bits == 0:
        return
    T, d = x.shape
    xd = torch.from_numpy(ref_xn).to(x.dtype).to(DEV)
    sd = None if s is None else torch.from_numpy(s).to(DEV)
    own_c, own_s = _codes_for(T, d, a_bits)
    own_c, own_s = own_c[:T], own_s[:T]
    if a_bits == 4:
        ref_c, ref_s = M.mx4_quant(M.smooth(ref_xn, s, False))
        c = M.unpack(codes.cpu().numpy())
        assert np.array_equal(np.where((c & 7) == 0, 0, c), np.where((ref_c & 7) == 0, 0, ref_c))
        L.qe_mx4_quant(xd, sd, own_c, own_s)
    else:
        ref_c, ref_s = O.quant_act(ref_xn, s, a_bits)
        assert np.array_equal(codes.cpu().numpy(), ref_c)
        L.qe_quant_act(xd, sd, a_bits, own_c, own_s)
    assert np.array_equal(scales.cpu().numpy(), ref_s)
    if a_bits != 4:
        assert torch.equal(codes, own_c)
    assert torch.equal(scales, own_s)


@pytest.mark.parametrize("a_bits", [0, 4, 6, 8])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,d", [(1, 32), (1, 1536), (3, 4096), (37, 544), (5, 8192), (2, 32768), (300, 256), (7, 18944)])
def test_norm(L, T, d, dtype, a_bits):
    x, r, w, s = _inputs(T, d, dtype)
    for res in (r, None):
        for sm in ([s, None] if a_bits else [None]):
            _check(L, x, res, w, sm, a_bits, _run(L, x, res, w, sm, a_bits))


@pytest.mark.parametrize("d", [8, 24, 520, 2056, 13000])
@pytest.mark.parametrize("a_bits", [0, 8])
def test_norm_widths_of_eight(L, d, a_bits):
    x, r, w, s = _inputs(11, d, torch.bfloat16)
    s = s if a_bits else None
    _check(L, x, r, w, s, a_bits, _run(L, x, r, w, s, a_bits))


@pytest.mark.parametrize("want_h,want_xn,a_bits", [(True, False, 0), (False, True, 0), (False, False, 4), (False, False, 8),
                                                   (True, False, 8), (False, True, 6)])
def test_outputs_left_out(L, want_h, want_xn, a_bits):
    x, r, w, s = _inputs(9, 1024, torch.bfloat16)
    s = s if a_bits else None
    _check(L, x, r, w, s, a_bits, _run(L, x, r, w, s, a_bits, want_h=want_h, want_xn=want_xn))


def test_mixed_weight_type(L):
    x, r, w, s = _inputs(6, 768, torch.bfloat16)
    w32 = w.float() + 1e-4
    _check(L, x, r, w32, s, 8, _run(L, x, r, w32, s, 8))
    x, r, w, s = _inputs(6, 768, torch.float32)
    wb = w.to(torch.bfloat16)
    _check(L, x, r, wb, s, 4, _run(L, x, r, wb, s, 4))


def test_extreme_rows(L):
    """Zero rows (codes 0, scale 0), squares beyond float32, and rows under eps."""
    d = 512
    x, r, w, s = _inputs(8, d, torch.float32)
    x[0], r[0] = 0.0, 0.0
    x[1], r[1] = x[1] * 1e25, r[1] * 1e25
    x[2], r[2] = x[2] * 1e-30, r[2] * 1e-30
    x[3, 1:], r[3] = 0.0, 0.0
    for a_bits in (4, 6, 8):
        got = _run(L, x, r, w, s, a_bits)
        _check(L, x, r, w, s, a_bits, got)
        assert not bool(got[1][0].any()) and not bool(got[2][0].any())
        if a_bits != 4:
            assert float(got[3][0]) == 0.0


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("d", [1536, 8192])
def test_in_place(L, d, dtype):
    """h and xn may be x or the residual itself."""
    x, r, w, s = _inputs(13, d, dtype)
    h, xn, c, sc = _run(L, x, r, w, s, 8)
    for hx in ("h is x, xn is res", "h is res, xn is x"):
        a, b = x.to(DEV), r.to(DEV)
        codes, scales = _codes_for(13, d, 8)
        oh, ox = (a, b) if hx.startswith("h is x") else (b, a)
        L.qe_add_rmsnorm(a, b, w.to(DEV), 1e-6, h=oh, xn=ox, smooth=torch.from_numpy(s).to(DEV), a_bits=8, codes=codes[:13],
                         scales=scales[:13])
        assert torch.equal(oh, h) and torch.equal(ox, xn) and torch.equal(codes[:13], c) and torch.equal(scales[:13], sc)


def test_many_rows(L):
    """More rows than one pass of the GPU holds."""
    x, r, w, s = _inputs(20000, 64, torch.bfloat16)
    _check(L, x, r, w, s, 4, _run(L, x, r, w, s, 4))
