"""Argument checks of the microscaled 4-bit and norm entry points (no GPU needed: every refused call
returns before anything is enqueued), and of their bindings."""

import ctypes

import pytest
import torch

P = 4096  # a 16-byte aligned address that no refused call reads


@pytest.fixture(scope="module")
def L():
    from quantized_linear_moe_amd import _libqe
    return _libqe


def _lin(L, **kw):
    a = dict(d_in=256, d_out=512, w_bits=4, a_bits=4, r_shared=8, n_routed=4, r_routed=8)
    a.update(kw)
    lin = L.make_linear(**a)
    lin.prep = P
    return lin


def test_quant_refusals(L):
    q = L.raw_library().qe_mx4_quant
    good = [P, 1, P, 0, 4, 256, P, P, None]
    for at, bad, want in [(1, 2, L.QE_ERR_INVALID_ARG), (3, 2, L.QE_ERR_INVALID_ARG), (3, -1, L.QE_ERR_INVALID_ARG),
                          (4, -1, L.QE_ERR_INVALID_ARG), (5, 0, L.QE_ERR_INVALID_ARG), (5, -32, L.QE_ERR_INVALID_ARG),
                          (5, 48, L.QE_ERR_UNSUPPORTED), (5, 8, L.QE_ERR_UNSUPPORTED), (0, None, L.QE_ERR_INVALID_ARG),
                          (6, None, L.QE_ERR_INVALID_ARG), (7, None, L.QE_ERR_INVALID_ARG), (0, P + 2, L.QE_ERR_ALIGNMENT),
                          (2, P + 4, L.QE_ERR_ALIGNMENT), (6, P + 8, L.QE_ERR_ALIGNMENT), (7, P + 1, L.QE_ERR_ALIGNMENT)]:
        args = list(good)
        args[at] = bad
        assert q(*args) == want, (at, bad)
    assert q(None, 1, None, 0, 0, 256, None, None, None) == L.QE_OK  # no tokens


def test_dequant_refusals(L):
    q = L.raw_library().qe_mx4_dequant
    good = [P, P, 4, 256, P, 1, None]
    for at, bad, want in [(5, 3, L.QE_ERR_INVALID_ARG), (2, -1, L.QE_ERR_INVALID_ARG), (3, 0, L.QE_ERR_INVALID_ARG),
                          (3, 40, L.QE_ERR_UNSUPPORTED), (0, None, L.QE_ERR_INVALID_ARG), (1, None, L.QE_ERR_INVALID_ARG),
                          (4, None, L.QE_ERR_INVALID_ARG), (0, P + 4, L.QE_ERR_ALIGNMENT), (4, P + 2, L.QE_ERR_ALIGNMENT)]:
        args = list(good)
        args[at] = bad
        assert q(*args) == want, (at, bad)
    assert q(None, None, 0, 256, None, 1, None) == L.QE_OK


def test_norm_refusals(L):
    f = L.raw_library().qe_add_rmsnorm
    # x res x_dtype weight w_dtype eps T d h xn smooth a_bits codes scales stream
    good = [P, P, 1, P, 1, 1e-6, 4, 256, 2 * P, 3 * P, P, 4, P, P, None]
    bad = [({2: 2}, "INVALID_ARG"), ({4: -1}, "INVALID_ARG"), ({5: 0.0}, "INVALID_ARG"), ({5: -1.0}, "INVALID_ARG"),
           ({5: float("nan")}, "INVALID_ARG"), ({5: float("inf")}, "INVALID_ARG"), ({6: -1}, "INVALID_ARG"),
           ({7: 0}, "INVALID_ARG"), ({11: 16}, "INVALID_ARG"), ({11: 5}, "INVALID_ARG"), ({7: 264}, "UNSUPPORTED"),
           ({7: 260, 11: 8}, "UNSUPPORTED"), ({7: 32800}, "UNSUPPORTED"), ({0: None}, "INVALID_ARG"),
           ({3: None}, "INVALID_ARG"), ({12: None}, "INVALID_ARG"), ({13: None}, "INVALID_ARG"),
           ({11: 0}, "INVALID_ARG"), ({11: 0, 12: None, 13: None}, "INVALID_ARG"),  # a smoothing vector without codes
           ({8: None, 9: None, 10: None, 11: 0, 12: None, 13: None}, "INVALID_ARG"),  # nothing asked for
           ({8: 3 * P}, "INVALID_ARG"),  # h and xn one buffer
           ({0: P + 2}, "ALIGNMENT"), ({1: P + 2}, "ALIGNMENT"), ({3: P + 8}, "ALIGNMENT"), ({8: 2 * P + 4}, "ALIGNMENT"),
           ({9: 3 * P + 4}, "ALIGNMENT"), ({10: P + 4}, "ALIGNMENT"), ({12: P + 4}, "ALIGNMENT"), ({13: P + 4}, "ALIGNMENT")]
    for change, want in bad:
        args = list(good)
        for at, v in change.items():
            args[at] = v
        assert f(*args) == getattr(L, "QE_ERR_" + want), change
    args = list(good)
    args[0] = args[3] = None
    args[6] = 0
    assert f(*args) == L.QE_OK


def test_prepare_and_gemm_refusals(L):
    lib = L.raw_library()
    lin = _lin(L)
    ref = ctypes.byref
    good = [ref(lin), P, P, None, P, P, P, P, P, P, None]
    assert lib.qe_mx4_prepare(ref(_lin(L, a_bits=8)), *good[1:]) == L.QE_ERR_INVALID_ARG
    assert lib.qe_mx4_prepare(ref(_lin(L, w_bits=3)), *good[1:]) == L.QE_ERR_UNSUPPORTED
    assert lib.qe_mx4_prepare(ref(_lin(L, d_in=192)), *good[1:]) == L.QE_ERR_UNSUPPORTED
    for at, bad, want in [(1, None, L.QE_ERR_INVALID_ARG), (2, None, L.QE_ERR_INVALID_ARG), (4, None, L.QE_ERR_INVALID_ARG),
                          (8, None, L.QE_ERR_INVALID_ARG), (9, None, L.QE_ERR_INVALID_ARG), (2, P + 4, L.QE_ERR_ALIGNMENT),
                          (3, P + 4, L.QE_ERR_ALIGNMENT), (5, P + 2, L.QE_ERR_ALIGNMENT)]:
        args = list(good)
        args[at] = bad
        assert lib.qe_mx4_prepare(*args) == want, (at, bad)

    for T in (1, 64, 65, 4096):
        need = L.qe_workspace_bytes(lin, T)
        good = [ref(lin), P, P, T, P, P, P, None, P, P, need, None]
        assert lib.qe_mx4_gemm(ref(_lin(L, a_bits=6)), *good[1:]) in (L.QE_ERR_INVALID_ARG, L.QE_ERR_WORKSPACE)
        for at, bad, want in [(1, None, L.QE_ERR_INVALID_ARG), (2, None, L.QE_ERR_INVALID_ARG), (3, -1, L.QE_ERR_INVALID_ARG),
                              (5, None, L.QE_ERR_INVALID_ARG), (6, None, L.QE_ERR_INVALID_ARG), (8, None, L.QE_ERR_INVALID_ARG),
                              (9, None, L.QE_ERR_WORKSPACE), (10, need - 1, L.QE_ERR_WORKSPACE), (1, P + 8, L.QE_ERR_ALIGNMENT),
                              (2, P + 4, L.QE_ERR_ALIGNMENT), (4, P + 2, L.QE_ERR_ALIGNMENT), (7, P + 4, L.QE_ERR_ALIGNMENT),
                              (8, P + 4, L.QE_ERR_ALIGNMENT)]:
            args = list(good)
            args[at] = bad
            assert lib.qe_mx4_gemm(*args) == want, (T, at, bad)
    assert lib.qe_mx4_gemm(ref(lin), None, None, 0, None, None, None, None, None, None, 0, None) == L.QE_OK
    # corrections that the linear does not have
    plain = _lin(L, r_shared=0, n_routed=0, r_routed=0)
    need = L.qe_workspace_bytes(plain, 4)
    assert lib.qe_mx4_gemm(ref(plain), P, P, 4, P, None, None, None, P, P, need, None) == L.QE_ERR_INVALID_ARG
    assert lib.qe_mx4_gemm(ref(plain), P, P, 4, None, P, P, None, P, P, need, None) == L.QE_ERR_INVALID_ARG


def test_integer_code_calls_refuse_microscaled_linears(L):
    lib = L.raw_library()
    lin = _lin(L)
    ref, need = ctypes.byref, L.qe_workspace_bytes(lin, 32)
    assert lib.qe_prepare(ref(lin), P, P, None, P, P, P, P, P, P, None) == L.QE_ERR_UNSUPPORTED
    assert lib.qe_wq_gemm(ref(lin), P, P, None, 1, 32, None, None, None, None, P, None, P, need, None) == \
        L.QE_ERR_UNSUPPORTED
    assert lib.qe_linear_prologue(ref(lin), P, 1, 32, P, P, P, P, P, None, P, need, None) == L.QE_ERR_UNSUPPORTED
    arr = lambda v: (ctypes.c_void_p * 1)(v)  # noqa: E731
    lins = (ctypes.POINTER(L.qe_linear) * 1)(ctypes.pointer(lin))
    wsb = (ctypes.c_size_t * 1)(need)
    assert lib.qe_group_prologue(lins, 1, P, 1, 32, arr(P), arr(P), arr(P), arr(P), arr(P), arr(None), arr(P), wsb,
                                 None) == L.QE_ERR_UNSUPPORTED
    assert lib.qe_group_gemm(lins, 1, arr(P), arr(P), 32, arr(None), arr(None), arr(None), arr(None), arr(P), arr(P),
                             wsb, None) == L.QE_ERR_UNSUPPORTED


@pytest.mark.parametrize("d_out", [16, 48, 256, 29568])
@pytest.mark.parametrize("d_in", [128, 1536, 29568])
def test_sizes_of_microscaled_linears(L, d_in, d_out):
    lin = L.make_linear(d_in, d_out, 4, 4, 0, 0, 0)
    out32 = (d_out + 31) // 32 * 32
    assert L.qe_prepared_bytes(lin) >= out32 * d_in // 2 + out32 * d_in // 32
    last = 0
    for T in (0, 1, 32, 33, 64, 65, 200, 4096):
        b = L.qe_workspace_bytes(lin, T)
        assert b >= T * d_in // 2 + T * d_in // 32
        last = b
    macs, _, byts = L.qe_linear_cost(lin, 8, 0, 2)
    assert macs == 8.0 * d_in * d_out
    assert byts == 8 * d_in * 2 + d_in * d_out * 17 / 32 + d_in * 4 + 8 * d_out * 4


def test_sizes_past_the_tiles_are_refused(L):
    """Tile ends are 32-bit numbers: 2^30 tokens or channels are the most that a microscaled linear takes."""
    lib = L.raw_library()
    lin, ref = _lin(L, r_shared=0, n_routed=0, r_routed=0), ctypes.byref
    assert lib.qe_workspace_bytes(ref(lin), 2 ** 30) > 2 ** 30
    for T in (2 ** 30 + 1, 2 ** 31 - 1):
        assert lib.qe_workspace_bytes(ref(lin), T) == 0
        big = 2 ** 62
        assert lib.qe_mx4_gemm(ref(lin), P, P, T, None, None, None, None, P, P, big, None) == L.QE_ERR_UNSUPPORTED
        assert lib.qe_linear_forward(ref(lin), P, 1, T, P, None, P, big, None) == L.QE_ERR_UNSUPPORTED
        assert lib.qe_linear_forward_noalloc(ref(lin), P, 1, T, P, None, None) == L.QE_ERR_WORKSPACE
    wide = _lin(L, d_out=2 ** 30 + 16, r_shared=0, n_routed=0, r_routed=0)
    assert lib.qe_prepared_bytes(ref(wide)) == 0
    assert lib.qe_mx4_prepare(ref(wide), P, P, None, None, None, None, None, None, P, None) == L.QE_ERR_UNSUPPORTED


def test_bindings_refuse_before_the_library_is_called(L):
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    codes, scales = torch.zeros(4, 32, dtype=torch.uint8), torch.zeros(4, 2, dtype=torch.uint8)
    with pytest.raises(ValueError, match="device tensors"):
        L.qe_mx4_quant(x, None, codes, scales)
    with pytest.raises(ValueError, match="codes must have shape"):
        L.qe_mx4_quant(x, None, scales, scales)
    with pytest.raises(TypeError, match="scales must be"):
        L.qe_mx4_dequant(codes, scales.int(), x)
    with pytest.raises(ValueError, match="contiguous"):
        L.qe_mx4_dequant(codes, torch.zeros(2, 4, dtype=torch.uint8).t(), x)
    with pytest.raises(TypeError, match="res must be"):
        L.qe_add_rmsnorm(x, x.float(), x[0], 1e-6, h=x)
    with pytest.raises(ValueError, match="weight must have shape"):
        L.qe_add_rmsnorm(x, x, x, 1e-6, h=x)
    lin = L.make_linear(64, 64, 4, 4, 0, 0, 0)
    with pytest.raises(TypeError, match="y must be"):
        L.qe_mx4_gemm(lin, codes, scales, None, None, None, x, codes)
