"""The forward of routed microscaled linears where one tile of the product holds every token, and on both sides
of that border.

Past the one-launch prologue the codes of bf16 tokens are written as the product's tiles in expert order, so the
product has to be given that order whatever the token count: without it a token gets another token's main product.
The shapes give tiles of 128 and 256 tokens, split and unsplit sums (tests/test_mx4_workspace.py pins that on the
CPU); the checks are those of test_gpu_mx4_forward.py, whose docstring derives their tolerances.
"""

import pytest
import torch

import test_gpu_mx4_forward as forward

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF = torch.bfloat16

SHAPES = [  # T, d_in, d_out, r_s, n_r, r_r, x
    (70, 29568, 6160, 0, 8, 16, BF), (128, 29568, 8192, 32, 8, 32, BF), (129, 29568, 8192, 32, 8, 32, BF),
    (65, 16384, 24592, 64, 16, 64, BF), (100, 8320, 24592, 8, 3, 8, BF), (200, 1024, 32784, 32, 8, 32, BF),
    (256, 1024, 32784, 16, 4, 64, BF), (257, 1024, 32784, 16, 4, 64, BF), (180, 8320, 32784, 0, 2, 8, BF),
]


@pytest.fixture(scope="module")
def Q():
    import quantized_linear_moe_amd as q
    return q


@pytest.mark.parametrize("shape", SHAPES, ids=forward.ids)
def test_codes(Q, shape):
    forward.test_codes(Q, shape)


@pytest.mark.parametrize("shape", SHAPES, ids=forward.ids)
def test_routes_and_corrections(Q, shape):
    forward.test_routes_and_corrections(Q, shape)


@pytest.mark.parametrize("shape", [SHAPES[i] for i in (0, 4, 5)], ids=forward.ids)
def test_graph_replays(Q, shape):
    forward.test_graph_replays(Q, shape)


@pytest.mark.parametrize("shape", [(100, 8320, 24592, 8, 3, 8, BF), (200, 1024, 32784, 32, 8, 32, BF)], ids=forward.ids)
def test_other_entry_points(Q, shape):
    """The allocation-free, grouped and top-2 forwards of the same linear: with B_s = B_r = 0 each is the product of
    qe_mx4_quant's codes, bit for bit."""
    L = Q.libqe
    T, d_in, d_out = shape[:3]
    rng, x, p = forward._case(shape)
    for k in ("B_s", "B_r"):
        p[k] = torch.zeros_like(p[k])
    w = torch.from_numpy(rng.integers(0, 256, (d_out, d_in // 2), dtype="uint8")).to(DEV)
    ws = torch.from_numpy(rng.integers(118, 124, (d_out, d_in // 32), dtype="uint8")).to(DEV)
    layer = forward._layer(Q, p, w, ws)
    codes = torch.empty(T, d_in // 2, dtype=torch.uint8, device=DEV)
    scales = torch.empty(T, d_in // 32, dtype=torch.uint8, device=DEV)
    L.qe_mx4_quant(x, torch.from_numpy(p["s"]).to(DEV), codes, scales)
    ref = torch.empty(T, d_out, device=DEV)
    L.qe_mx4_gemm(layer.lin, codes, scales, None, None, None, ref, layer.workspace(T))
    nan = lambda: torch.full((T, d_out), float("nan"), device=DEV)  # noqa: E731
    routes = lambda: torch.empty(T, dtype=torch.int32, device=DEV)  # noqa: E731

    y = nan()
    assert L.qe_workspace_bytes(layer.lin, T) <= L.qe_noalloc_scratch_bytes()
    L.qe_linear_forward_noalloc(layer.lin, x, y, routes())
    assert torch.equal(y, ref)

    ys = [nan(), nan()]
    L.qe_group_forward([layer.lin, layer.lin], x, ys, [routes(), routes()], [layer.workspace(T), layer.workspace(T)])
    assert torch.equal(ys[0], ref) and torch.equal(ys[1], ref)

    y = nan()
    ws2 = torch.empty(L.qe_top2_workspace_bytes(layer.lin, T), dtype=torch.uint8, device=DEV)
    L.qe_linear_forward_top2(layer.lin, x, y, routes(), routes(), ws2)
    assert torch.equal(y, ref)
