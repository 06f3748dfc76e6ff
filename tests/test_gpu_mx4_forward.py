"""The forward of microscaled linears over the shapes that choose how its codes, routes and adapter inputs are
made: in one launch per row (few tokens, up to 8192 channels), with the projections' finish, in two passes over
x (codes as rows or straight as the product's tiles), or apart (float32 x).

(1) Codes: with B_s = B_r = 0 the corrections add exact zeros at the end of every sum, so the forward is the
product of qe_mx4_quant's codes, bit for bit.  (2) Routes, u and v: with W = 0 the forward is the corrections
alone.  u is a float32 sum of d_in terms in any order (each addition off by at most 2^-23 of a partial sum,
which the magnitudes bound) rounded to bf16 (2^-8), and so is v; the last sum is float32 again:
|dy| <= 2^-8 (|u||B_s| + |v||B_e|) + 3 (d_in + 64) 2^-23 (|x||A||B| of both).
"""

import numpy as np
import pytest
import torch


pytestmark = pytest.mark.gpu
DEV = "cuda"
BF, F32 = torch.bfloat16, torch.float32

SHAPES = [  # T, d_in, d_out, r_s, n_r, r_r, x
    (1, 8320, 64, 32, 8, 32, BF), (16, 4224, 48, 0, 4, 64, F32), (16, 8320, 48, 64, 0, 0, BF), (9, 640, 32, 0, 0, 0, BF),
    (3, 1536, 48, 32, 8, 32, BF), (5, 128, 16, 8, 2, 1, BF), (100, 2048, 80, 64, 16, 64, BF), (64, 8192, 48, 0, 4, 8, BF),
    (20, 8320, 64, 32, 8, 32, BF), (250, 8320, 64, 0, 4, 64, BF), (130, 1024, 96, 16, 3, 8, BF), (300, 1024, 96, 33, 2, 48, BF),
    (300, 1152, 96, 8, 4, 8, BF), (300, 640, 64, 64, 0, 0, BF), (300, 640, 64, 32, 8, 32, F32), (17, 8320, 64, 0, 0, 0, BF),
    (4101, 1024, 4112, 32, 8, 32, BF), (4097, 1024, 4112, 0, 16, 64, BF), (4100, 1024, 4112, 16, 0, 0, BF),
    (4127, 1024, 4112, 32, 8, 32, F32), (4100, 1024, 4112, 0, 0, 0, BF), (2, 384, 48, 64, 16, 64, F32),
]
ids = lambda s: "x".join(str(v).replace("torch.", "") for v in s)  # noqa: E731


@pytest.fixture(scope="module")
def Q():
    import quantized_linear_moe_amd as q
    return q


def _case(shape):
    T, d_in, d_out, r_s, n_r, r_r, dt = shape
    rng = np.random.default_rng(sum(shape[:6]))
    bf = lambda *s: torch.from_numpy((0.05 * rng.standard_normal(s)).astype(np.float32)).to(BF)  # noqa: E731
    x = rng.standard_normal((T, d_in)).astype(np.float32)
    x[:, rng.integers(0, d_in, 3)] *= 30.0
    x[T // 2, : d_in // 2] = 0.0  # blocks of zeros
    p = dict(d_in=d_in, d_out=d_out, s=rng.uniform(0.5, 2.0, d_in).astype(np.float32))
    if r_s:
        p["A_s"], p["B_s"] = bf(d_in, r_s), bf(r_s, d_out)
    if n_r:
        p["A_r"], p["B_r"], p["R"] = bf(n_r, d_in, r_r), bf(n_r, r_r, d_out), bf(d_in, n_r)
    return rng, torch.from_numpy(x).to(dt).to(DEV), p


def _layer(Q, p, codes, scales):
    return Q.QELinear.from_params(p, 4, 4, device=DEV, packed=codes, w_scale=scales)


def _forward(Q, layer, x, d_out):
    """The forward in a workspace of NaN patterns, with sentinel rows behind y and the routes."""
    L, T = Q.libqe, x.shape[0]
    y = torch.full((T + 1, d_out), 77.0, device=DEV)
    e = torch.full((T + 1,), 77, dtype=torch.int32, device=DEV)
    ws = torch.full((L.qe_workspace_bytes(layer.lin, T),), 255, dtype=torch.uint8, device=DEV)
    L.qe_linear_forward(layer.lin, x, y, e, ws)
    torch.cuda.synchronize()
    assert bool((y[T] == 77.0).all()) and int(e[T]) == 77
    return y[:T], e[:T]


@pytest.mark.parametrize("shape", SHAPES, ids=ids)
def test_codes(Q, shape):
    L = Q.libqe
    T, d_in, d_out = shape[:3]
    rng, x, p = _case(shape)
    for k in ("B_s", "B_r"):
        if k in p:
            p[k] = torch.zeros_like(p[k])
    w = torch.from_numpy(rng.integers(0, 256, (d_out, d_in // 2)).astype(np.uint8)).to(DEV)
    ws = torch.from_numpy(rng.integers(118, 124, (d_out, d_in // 32)).astype(np.uint8)).to(DEV)
    layer = _layer(Q, p, w, ws)
    y, _ = _forward(Q, layer, x, d_out)
    codes = torch.empty(T, d_in // 2, dtype=torch.uint8, device=DEV)
    scales = torch.empty(T, d_in // 32, dtype=torch.uint8, device=DEV)
    L.qe_mx4_quant(x, torch.from_numpy(p["s"]).to(DEV), codes, scales)
    ref = torch.full_like(y, float("nan"))
    L.qe_mx4_gemm(layer.lin, codes, scales, None, None, None, ref, layer.workspace(T))
    assert torch.equal(y, ref)


@pytest.mark.parametrize("shape", [s for s in SHAPES if s[3] or s[4]], ids=ids)
def test_routes_and_corrections(Q, shape):
    T, d_in, d_out, r_s, n_r, _, _ = shape
    _, x, p = _case(shape)
    zero = lambda n: torch.zeros(d_out, n, dtype=torch.uint8, device=DEV)  # noqa: E731
    y, e = _forward(Q, _layer(Q, p, zero(d_in // 2), zero(d_in // 32)), x, d_out)
    xb = x.to(BF).double().cpu().numpy()
    ref, value, terms = (np.zeros((T, d_out)) for _ in range(3))

    def add(rows, A, B):
        A, B = A.double().numpy(), B.double().numpy()
        u = xb[rows] @ A
        ref[rows] += u @ B
        value[rows] += np.abs(u) @ np.abs(B)
        terms[rows] += (np.abs(xb[rows]) @ np.abs(A)) @ np.abs(B)

    if r_s:
        add(np.arange(T), p["A_s"], p["B_s"])
    if n_r:
        e = e.cpu().numpy()
        scores = xb @ p["R"].double().numpy()
        assert e.min() >= 0 and e.max() < n_r
        # the route is the smallest score, up to the float32 sums' error
        slack = 2 * d_in * 2.0 ** -23 * (np.abs(xb) @ np.abs(p["R"].double().numpy())).max(axis=1)
        assert np.all(scores[np.arange(T), e] <= scores.min(axis=1) + slack)
        for k in range(n_r):
            add(np.flatnonzero(e == k), p["A_r"][k], p["B_r"][k])
    tol = 2.0 ** -8 * value + 3 * (d_in + 64) * 2.0 ** -23 * terms
    err = np.abs(y.double().cpu().numpy() - ref)
    assert np.all(err <= tol), float((err / np.maximum(tol, 1e-30)).max())


@pytest.mark.parametrize("shape", [SHAPES[i] for i in (0, 1, 2, 4, 6, 8, 9, 12, 16, 18, 19)], ids=ids)
def test_graph_replays(Q, shape):
    """Captured once and replayed on new inputs, between eager forwards of the same linear in the same workspace."""
    L = Q.libqe
    T, d_in, d_out = shape[:3]
    rng, x0, p = _case(shape)
    w = torch.from_numpy(rng.integers(0, 256, (d_out, d_in // 2)).astype(np.uint8)).to(DEV)
    layer = _layer(Q, p, w, torch.from_numpy(rng.integers(118, 124, (d_out, d_in // 32)).astype(np.uint8)).to(DEV))
    ws = layer.workspace(T)

    def run(x):
        y = torch.empty(T, d_out, device=DEV)
        e = torch.zeros(T, dtype=torch.int32, device=DEV)
        L.qe_linear_forward(layer.lin, x, y, e, ws)
        return y, e

    inputs = [x0, -x0, x0.flip(0).contiguous(), 0.5 * x0]
    eager = [run(x) for x in inputs]
    x = x0.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y, e = run(x)
    for i in (1, 2, 0, 3, 3):
        x.copy_(inputs[i])
        y.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, eager[i][0]) and torch.equal(e, eager[i][1])
        again = run(inputs[(i + 1) % 4])
        assert torch.equal(again[0], eager[(i + 1) % 4][0])
