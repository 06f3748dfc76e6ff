"""The microscaled operators at sizes whose tiles or offsets leave the usual range: more token tiles than one
column of channels can share out, and tensors of more than 2^31 elements.

Every row of these operators depends on its own input row alone, so the rows of a large call are compared bit
for bit with those of a small call on the same rows.  For the product, whose kernels order their sums
differently, the operands make every sum exact: codes times scales of 1/2, 1 and 2 are multiples of 2^-4,
1024 products of at most 144 and 64 integers of at most 4 stay below 2^18, and 22 bits fit float32.
"""

import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module")
def Q():
    import quantized_linear_moe_amd as q
    return q


def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _product(Q, T, d_in, d_out, y_dtype, rows):
    """The product of T tokens, and of the tokens `rows` alone."""
    L, g = Q.libqe, _gen(T + d_out)
    ints = lambda lo, hi, *shape, dtype: torch.randint(lo, hi, shape, generator=g, device=DEV, dtype=dtype)  # noqa: E731
    bf = lambda *shape: ints(-2, 3, *shape, dtype=torch.int32).to(torch.bfloat16)  # noqa: E731
    layer = Q.QELinear.from_params(
        dict(d_in=d_in, d_out=d_out, A_s=bf(d_in, 32), B_s=bf(32, d_out), A_r=bf(4, d_in, 32), B_r=bf(4, 32, d_out),
             R=bf(d_in, 4)), 4, 4, device=DEV, packed=ints(0, 256, d_out, d_in // 2, dtype=torch.uint8),
        w_scale=ints(126, 129, d_out, d_in // 32, dtype=torch.uint8))
    layer.lin.y_dtype = L.QE_BF16 if y_dtype == torch.bfloat16 else L.QE_F32
    args = (ints(0, 256, T, d_in // 2, dtype=torch.uint8), ints(126, 129, T, d_in // 32, dtype=torch.uint8), bf(T, 32),
            bf(T, 32), ints(0, 4, T, dtype=torch.int32))
    out = []
    for part in (args, tuple(a[rows].contiguous() for a in args)):
        y = torch.full((part[0].shape[0], d_out), float("nan"), dtype=y_dtype, device=DEV)
        L.qe_mx4_gemm(layer.lin, *part, y, layer.workspace(part[0].shape[0]))
        out.append(y)
    torch.cuda.synchronize()
    return out


@pytest.mark.parametrize("T,d_out", [(66000, 256), (66000, 16), (40000, 512)])
def test_more_token_tiles_than_a_round(Q, T, d_out):
    rows = torch.cat([torch.arange(0, 40), torch.arange(T // 2, T // 2 + 40), torch.arange(T - 40, T)]).to(DEV)
    y, few = _product(Q, T, 1024, d_out, torch.float32, rows)
    assert not bool(torch.isnan(y).any())
    assert torch.equal(y[rows], few)


def test_product_past_31_bits(Q):
    T, d_out = 70016, 30736
    assert T * d_out > 2 ** 31
    rows = torch.cat([torch.arange(0, 30), torch.arange(T - 30, T)]).to(DEV)
    y, few = _product(Q, T, 1024, d_out, torch.bfloat16, rows)
    assert torch.equal(y[rows], few)


def test_quantization_past_31_bits(Q):
    L = Q.libqe
    T, d = 70016, 32768
    assert T * d > 2 ** 31
    g = _gen(3)
    x = torch.randn(T, d, generator=g, device=DEV, dtype=torch.bfloat16)
    s = 0.5 + torch.rand(d, generator=g, device=DEV)
    codes = torch.empty(T, d // 2, dtype=torch.uint8, device=DEV)
    scales = torch.empty(T, d // 32, dtype=torch.uint8, device=DEV)
    L.qe_mx4_quant(x, s, codes, scales)
    back = torch.full_like(x, float("nan"))
    L.qe_mx4_dequant(codes, scales, back)
    for r in (slice(0, 5), slice(T - 5, T)):
        c, e = torch.empty_like(codes[r]), torch.empty_like(scales[r])
        L.qe_mx4_quant(x[r].contiguous(), s, c, e)
        b = torch.empty_like(x[r])
        L.qe_mx4_dequant(c, e, b)
        assert torch.equal(codes[r], c) and torch.equal(scales[r], e) and torch.equal(back[r], b)


@pytest.mark.parametrize("a_bits", [4, 8])
def test_norm_past_31_bits(Q, a_bits):
    L = Q.libqe
    T, d = 70016, 32768
    g = _gen(a_bits)
    x = torch.randn(T, d, generator=g, device=DEV, dtype=torch.bfloat16)
    w = 0.5 + torch.rand(d, generator=g, device=DEV)

    def run(x):
        n = x.shape[0]
        xn = torch.empty_like(x)
        codes = torch.empty(n, d // 2 if a_bits == 4 else d, dtype=torch.uint8 if a_bits == 4 else torch.int8, device=DEV)
        scales = torch.empty((n, d // 32) if a_bits == 4 else n, dtype=torch.uint8 if a_bits == 4 else torch.float32, device=DEV)
        L.qe_add_rmsnorm(x, None, w, 1e-6, xn=xn, a_bits=a_bits, codes=codes, scales=scales)
        return xn, codes, scales

    whole = run(x)
    for r in (slice(0, 5), slice(T - 5, T)):
        for a, b in zip(whole, run(x[r].contiguous())):
            assert torch.equal(a[r], b)
