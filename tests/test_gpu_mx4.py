"""GPU parity of the microscaled 4-bit operators against the float64 oracle.

Quantization decides codes by exact comparisons, so codes and scales are compared bit for bit.

The product is compared in two ways.  (1) Exactly: codes at random, scales 2^-2 .. 2^2 and small integer
adapters make every product a multiple of 2^-6 and every partial sum, in any order, smaller than 2^18, so
float32 holds each of them exactly and y has one right value (bf16 outputs: its rounding).  The bound on the
partial sums is checked: they lie between the sum of the negative and that of the positive terms.  (2) On natural values, within the error of a
float32 sum in any order: each of the n <= d_in + ranks additions is off by at most one step (2^-23: half
a step for rounding, a whole one where the matrix core truncates) of a partial sum that the sum of
magnitudes bounds, so |dy| <= n 2^-23 sum|terms|; bf16 outputs add half a step, 2^-8 |y|.
"""

import numpy as np
import pytest
import torch

import synth
from oracle import qe_mx4_oracle as M
from oracle import qe_oracle as O

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module")
def Q():
    import quantized_linear_moe_amd as q
    return q


def _dev(a, dtype=None):
    t = torch.from_numpy(np.ascontiguousarray(a))
    return (t if dtype is None else t.to(dtype)).to(DEV)


def _guarded(T, d, dtype):
    """A [T, d] buffer with 256 sentinel elements behind it, and a check that they still stand."""
    fill = 77 if not dtype.is_floating_point else -77.0
    buf = torch.full((T * d + 256,), fill, dtype=dtype, device=DEV)

    def check():
        assert bool((buf[T * d:] == fill).all()), "elements behind the last row were written"

    return buf[: T * d].view(T, d), check


# ------------------------------------------------------------------ quantization
def _mixed_rows(rng, T, d):
    """Rows of very different magnitude, zeros, denormals, exact ties and signed zeros."""
    x = (rng.standard_normal((T, d)) * np.exp2(rng.integers(-30, 30, (T, 1)))).astype(np.float32)
    x[:, rng.integers(0, d, 3)] = 0.0
    x[0, :32] = 0.0
    if T > 1:
        x[1] = rng.integers(-64, 65, d) * 0.125  # many exact halves between levels
    if T > 2:
        x[2] = np.ldexp(rng.standard_normal(d), -126 - rng.integers(0, 20)).astype(np.float32)
    if T > 3:
        x[3] = -0.0
    if T > 4:
        x[4] = np.float32(3.4e38) * rng.choice([-1.0, 1.0], d)
    return x


@pytest.mark.parametrize("how", ["none", "div", "mul"])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T,d", [(1, 32), (1, 29568), (7, 96), (64, 2048), (33, 2080), (5, 4128), (300, 160), (1025, 544)])
def test_quant_matches_oracle(Q, T, d, dtype, how):
    L = Q.libqe
    rng = np.random.default_rng(T * 31 + d)
    x = torch.from_numpy(_mixed_rows(rng, T, d)).to(dtype)
    if how != "none":
        x[4:5] = 1.0  # the largest float32 values times a factor are no longer finite
    s = None if how == "none" else rng.uniform(0.25, 4.0, d).astype(np.float32)
    codes, c1 = _guarded(T, d // 2, torch.uint8)
    scales, c2 = _guarded(T, d // 32, torch.uint8)
    L.qe_mx4_quant(x.to(DEV), None if s is None else _dev(s), codes, scales, multiply=how == "mul")
    torch.cuda.synchronize()
    c1(), c2()
    ref_c, ref_s = M.mx4_quant(M.smooth(x.float().numpy(), s, how == "mul"))
    assert np.array_equal(scales.cpu().numpy(), ref_s)
    got = M.unpack(codes.cpu().numpy())
    # the sign of a zero has no meaning: -0 may stand for 0
    zero = (got & 7) == 0
    assert np.array_equal(np.where(zero, 0, got), np.where((ref_c & 7) == 0, 0, ref_c))


def test_quant_extreme_factors(Q):
    """Factors and values outside the range of the reciprocal form of the division."""
    L = Q.libqe
    rng = np.random.default_rng(3)
    d = 256
    s = np.exp2(rng.uniform(-120, 120, d)).astype(np.float32)
    x = (rng.standard_normal((40, d)) * np.exp2(rng.uniform(-120, 120, (40, d)))).astype(np.float32)
    q = M.smooth(x, s, False)
    x[~np.isfinite(q)] = 0.0
    codes = torch.empty(40, d // 2, dtype=torch.uint8, device=DEV)
    scales = torch.empty(40, d // 32, dtype=torch.uint8, device=DEV)
    L.qe_mx4_quant(_dev(x), _dev(s), codes, scales)
    ref_c, ref_s = M.mx4_quant(M.smooth(x, s, False))
    assert np.array_equal(scales.cpu().numpy(), ref_s)
    got = M.unpack(codes.cpu().numpy())
    assert np.array_equal(np.where((got & 7) == 0, 0, got), np.where((ref_c & 7) == 0, 0, ref_c))


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
def test_non_finite_blocks(Q, bad):
    """The block that holds the value reads back as NaN and makes its token's outputs NaN; the others stay."""
    L = Q.libqe
    rng = np.random.default_rng(5)
    T, d = 70, 256
    x = torch.from_numpy(rng.standard_normal((T, d)).astype(np.float32))
    x[2, 100] = bad
    codes = torch.empty(T, d // 2, dtype=torch.uint8, device=DEV)
    scales = torch.empty(T, d // 32, dtype=torch.uint8, device=DEV)
    back = torch.empty(T, d, dtype=torch.float32, device=DEV)
    L.qe_mx4_quant(x.to(DEV), None, codes, scales)
    L.qe_mx4_dequant(codes, scales, back)
    nan = torch.isnan(back).cpu()
    assert bool(nan[2, 96:128].all()) and int(nan.sum()) == 32
    layer = Q.QELinear.from_params(dict(W_f=rng.standard_normal((48, d)).astype(np.float32)), 4, 4, device=DEV)
    for n in (T, 8):  # both kernels
        y = torch.empty(n, 48, dtype=torch.float32, device=DEV)
        L.qe_mx4_gemm(layer.lin, codes[:n].contiguous(), scales[:n].contiguous(), None, None, None, y, layer.workspace(n))
        nan = torch.isnan(y).cpu()
        assert bool(nan[2].all()) and int(nan.sum()) == 48


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T,d", [(1, 32), (9, 992), (130, 4096)])
def test_dequant_is_exact(Q, T, d, dtype):
    L = Q.libqe
    rng = np.random.default_rng(T + d)
    packed = rng.integers(0, 256, (T, d // 2)).astype(np.uint8)
    scales = rng.integers(4, 250, (T, d // 32)).astype(np.uint8)
    scales[0, 0] = 255
    out, check = _guarded(T, d, dtype)
    L.qe_mx4_dequant(_dev(packed), _dev(scales), out)
    check()
    ref = M.mx4_values(M.unpack(packed), scales).astype(np.float32)
    got = out.float().cpu().numpy()
    assert np.array_equal(got, ref, equal_nan=True)


def test_dequant_lowest_scales_round_to_nearest(Q):
    L = Q.libqe
    packed = np.tile(np.arange(16, dtype=np.uint8) * 17, 4).reshape(4, 16)
    for dtype in (torch.float32, torch.bfloat16):
        scales = np.arange(4, dtype=np.uint8).reshape(4, 1)
        out = torch.empty(4, 32, dtype=dtype, device=DEV)
        L.qe_mx4_dequant(_dev(packed), _dev(scales), out)
        ref = torch.from_numpy(M.mx4_values(M.unpack(packed), scales)).float().to(dtype)
        assert torch.equal(out.cpu(), ref)


# ------------------------------------------------------------------ product
def _exact_operand(rng, T, d):
    return M.pack(rng.integers(0, 16, (T, d)).astype(np.uint8)), rng.integers(125, 130, (T, d // 32)).astype(np.uint8)


def _layer(Q, w_packed, w_scales, d_in, d_out, r_s, n_r, r_r, rng, y_bf16=False):
    bf = lambda *shape: torch.from_numpy(rng.integers(-2, 3, shape).astype(np.float32)).to(torch.bfloat16)  # noqa: E731
    p = dict(d_in=d_in, d_out=d_out)
    if r_s:
        p["A_s"], p["B_s"] = bf(d_in, r_s), bf(r_s, d_out)
    if n_r:
        p["A_r"], p["B_r"], p["R"] = bf(n_r, d_in, r_r), bf(n_r, r_r, d_out), bf(d_in, n_r)
    layer = Q.QELinear.from_params(p, 4, 4, device=DEV, packed=_dev(w_packed), w_scale=_dev(w_scales))
    layer.lin.y_dtype = Q.libqe.QE_BF16 if y_bf16 else Q.libqe.QE_F32
    return layer, p


def _rows(rng, T, r, pad):
    u = np.zeros((T, pad), np.float32)
    u[:, :r] = rng.integers(-2, 3, (T, r))
    return u


SHAPES = [  # T, d_in, d_out, r_s, n_r, r_r
    (1, 128, 16, 0, 0, 0), (1, 2048, 1024, 8, 4, 8), (3, 384, 48, 32, 8, 32), (8, 29568, 80, 32, 8, 32),
    (16, 1152, 2064, 0, 16, 64), (32, 640, 400, 64, 0, 0), (33, 1024, 96, 8, 3, 48), (64, 896, 528, 33, 2, 1),
    (65, 128, 16, 0, 0, 0), (65, 2048, 272, 32, 8, 32), (127, 1280, 304, 0, 4, 16), (128, 512, 2064, 16, 8, 8),
    (200, 256, 1040, 64, 16, 64), (513, 1536, 256, 8, 4, 48), (1000, 640, 1552, 32, 8, 32), (2048, 256, 8208, 32, 8, 32),
    (4099, 128, 4112, 8, 4, 8), (40, 512, 25616, 32, 8, 32), (100, 8192, 3216, 32, 8, 32), (17, 8192, 528, 16, 4, 64),
    (257, 1152, 16400, 8, 16, 32), (4352, 1024, 4112, 32, 8, 32), (48, 1024, 4112, 64, 16, 64),
    (130, 1152, 32800, 32, 8, 32), (200, 8192, 12304, 8, 4, 32), (70, 29568, 6160, 0, 8, 16), (150, 14336, 5136, 32, 0, 0),
    (100, 1024, 65552, 8, 4, 8), (17, 1024, 65552, 0, 0, 0),
]


@pytest.mark.parametrize("y_bf16", [False, True])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s)))
def test_gemm_exact(Q, shape, y_bf16):
    L = Q.libqe
    T, d_in, d_out, r_s, n_r, r_r = shape
    rng = np.random.default_rng(sum(shape))
    a_c, a_s = _exact_operand(rng, T, d_in)
    w_c, w_s = _exact_operand(rng, d_out, d_in)
    layer, p = _layer(Q, w_c, w_s, d_in, d_out, r_s, n_r, r_r, rng, y_bf16)
    u = _rows(rng, T, r_s, L.rank_pad(r_s)) if r_s else None
    v = _rows(rng, T, r_r, L.rank_pad(r_r)) if n_r else None
    expert = rng.integers(0, n_r, T).astype(np.int32) if n_r else None
    av, wv = M.mx4_values(M.unpack(a_c), a_s), M.mx4_values(M.unpack(w_c), w_s)
    ref, mag = M.mx4_gemm(av, wv, None if u is None else u[:, :r_s], None if u is None else p["B_s"].float().numpy(),
                          None if v is None else v[:, :r_r], expert, None if v is None else p["B_r"].float().numpy())
    # any partial sum lies between the sum of the negative terms, (y - mag) / 2, and that of the positive ones,
    # (y + mag) / 2; multiples of 2^-6 below 2^18 are float32 values
    assert ((mag + np.abs(ref)) / 2).max() < 2.0 ** 18
    ref = torch.from_numpy(ref.astype(np.float32))
    ref = ref.to(torch.bfloat16) if y_bf16 else ref
    bf = lambda t: None if t is None else _dev(t, torch.bfloat16)  # noqa: E731
    order = None if expert is None else np.argsort(expert, kind="stable").astype(np.int32)
    for perm in ([None] if order is None else [None, order]):
        y, check = _guarded(T, d_out, ref.dtype)
        y.fill_(float("nan"))
        ws = torch.full((max(L.qe_workspace_bytes(layer.lin, T), 256),), 255, dtype=torch.uint8, device=DEV)
        L.qe_mx4_gemm(layer.lin, _dev(a_c), _dev(a_s), bf(u), bf(v), None if expert is None else _dev(expert), y, ws,
                      perm=None if perm is None else _dev(perm))
        torch.cuda.synchronize()
        check()
        bad = int((y.cpu() != ref).sum())
        assert bad == 0, f"{bad} of {ref.numel()} outputs differ (perm {perm is not None})"


@pytest.mark.parametrize("y_bf16", [False, True])
@pytest.mark.parametrize("T,d_in,d_out", [(1, 8192, 256), (24, 3584, 512), (150, 2048, 640), (700, 4096, 768)])
def test_gemm_natural_values(Q, T, d_in, d_out, y_bf16):
    L = Q.libqe
    rng = np.random.default_rng(T + d_in)
    r_s, n_r, r_r = 32, 8, 32
    x = rng.standard_normal((T, d_in)).astype(np.float32)
    x[:, rng.integers(0, d_in, 8)] *= 30.0
    a_c, a_s = M.mx4_quant(x)
    w_c, w_s = M.mx4_quant((0.02 * rng.standard_normal((d_out, d_in))).astype(np.float32))
    layer, p = _layer(Q, M.pack(w_c), w_s, d_in, d_out, r_s, n_r, r_r, rng, y_bf16)
    u = torch.from_numpy(rng.standard_normal((T, 32)).astype(np.float32)).to(torch.bfloat16)
    v = torch.from_numpy(rng.standard_normal((T, 32)).astype(np.float32)).to(torch.bfloat16)
    expert = rng.integers(0, n_r, T).astype(np.int32)
    ref, mag = M.mx4_gemm(M.mx4_values(a_c, a_s), M.mx4_values(w_c, w_s), u.double().numpy(), p["B_s"].double().numpy(),
                          v.double().numpy(), expert, p["B_r"].double().numpy())
    y = torch.empty(T, d_out, dtype=torch.bfloat16 if y_bf16 else torch.float32, device=DEV)
    L.qe_mx4_gemm(layer.lin, _dev(M.pack(a_c)), _dev(a_s), u.to(DEV), v.to(DEV), _dev(expert), y, layer.workspace(T))
    tol = (d_in + r_s + r_r) * 2.0 ** -23 * mag + (2.0 ** -8 * np.abs(ref) * (1 + 2.0 ** -8) if y_bf16 else 0.0)
    err = np.abs(y.double().cpu().numpy() - ref)
    assert np.all(err <= tol), float((err / tol).max())


def test_gemm_is_deterministic_and_clamps_experts(Q):
    L = Q.libqe
    rng = np.random.default_rng(9)
    T, d_in, d_out, n_r = 130, 1024, 144, 4
    a_c, a_s = _exact_operand(rng, T, d_in)
    w_c, w_s = _exact_operand(rng, d_out, d_in)
    layer, _ = _layer(Q, w_c, w_s, d_in, d_out, 0, n_r, 8, rng)
    v = _dev(_rows(rng, T, 8, 32), torch.bfloat16)
    e = rng.integers(-3, n_r + 3, T).astype(np.int32)
    outs = []
    for experts in (e, e, np.clip(e, 0, n_r - 1)):
        for n in (T, 20):
            y = torch.empty(n, d_out, dtype=torch.float32, device=DEV)
            L.qe_mx4_gemm(layer.lin, _dev(a_c[:n]), _dev(a_s[:n]), None, v[:n].contiguous(), _dev(experts[:n]), y,
                          layer.workspace(n))
            outs.append(y)
    for i in (2, 3, 4, 5):
        assert torch.equal(outs[i], outs[i % 2])
    assert torch.equal(outs[0][:20], outs[1])


# ------------------------------------------------------------------ the whole linear
def _oracle_forward(params, x, expert):
    """y of the microscaled QE linear in float64 with the given routes, and the terms' magnitudes."""
    s = params["s"]
    a = M.mx4_values(*M.mx4_quant(M.smooth(x.float().numpy(), s, False)))
    w = M.mx4_values(*M.mx4_quant(M.smooth(params["W_f"], s, True)))
    xb = x.to(torch.bfloat16).double().numpy()
    u = xb @ params["A_s"].double().numpy()
    v = np.stack([xb[t] @ params["A_r"][expert[t]].double().numpy() for t in range(len(expert))])
    return M.mx4_gemm(a, w, u, params["B_s"].double().numpy(), v, expert, params["B_r"].double().numpy())


@pytest.mark.parametrize("T", [1, 8, 64, 100, 700])
@pytest.mark.parametrize("cfg_name,lin_name", [("tiny", "lin"), ("qwen2vl_2b", "k"), ("qwen2vl_2b", "q")])
def test_linear_forward(Q, cfg_name, lin_name, T):
    """The adapter inputs u and v are rounded to bf16 (2^-8 relative each, on terms bounded by their
    magnitudes); the rest as for the product.  Routes agree away from near-ties."""
    L = Q.libqe
    cfg = synth.get_config(cfg_name)
    spec = next(l for l in cfg.linears if l.name == lin_name)
    params = synth.gen_linear(cfg, spec)
    x = synth.gen_activations(cfg, spec.stream, T=T)
    layer = Q.QELinear.from_params(params, 4, 4, device=DEV)
    e = torch.full((T,), -1, dtype=torch.int32, device=DEV)
    y = layer.forward(x.to(DEV), expert_out=e)
    expert = e.cpu().numpy()
    r = O.route(x.to(torch.bfloat16).float().numpy(), params["R"].float().numpy())
    near = r["margin"] < 1e-4 * r["margin_scale"]
    assert np.all((expert == r["expert"]) | near)
    ref, mag = _oracle_forward(params, x, expert)
    # float32 sums behind u and v (2^-23 d_in of their magnitudes), then bf16: 2^-8
    xb = np.abs(x.to(torch.bfloat16).double().numpy())
    um = xb @ np.abs(params["A_s"].double().numpy())
    vm = np.stack([xb[t] @ np.abs(params["A_r"][expert[t]].double().numpy()) for t in range(T)])
    _, adapter_mag = M.mx4_gemm(np.zeros((T, 1)), np.zeros((spec.d_out, 1)), um, params["B_s"].double().numpy(), vm, expert,
                                params["B_r"].double().numpy())
    n = spec.d_in + 64
    xs = x.to(torch.bfloat16).double().numpy()
    uv = np.abs(xs @ params["A_s"].double().numpy())
    vv = np.abs(np.stack([xs[t] @ params["A_r"][expert[t]].double().numpy() for t in range(T)]))
    _, value_mag = M.mx4_gemm(np.zeros((T, 1)), np.zeros((spec.d_out, 1)), uv, params["B_s"].double().numpy(), vv, expert,
                              params["B_r"].double().numpy())
    tol = n * 2.0 ** -23 * (mag + 2 * adapter_mag) + 2.0 ** -8 * value_mag
    err = np.abs(y.double().cpu().numpy() - ref)
    assert np.all(err <= tol), float((err / tol).max())
    # the same call without a workspace, and as a group of one
    y2 = torch.empty_like(y)
    L.qe_linear_forward_noalloc(layer.lin, x.to(DEV), y2, None)
    y3 = torch.empty_like(y)
    L.qe_group_forward([layer.lin], x.to(DEV), [y3], None, [layer.workspace(T)])
    assert torch.equal(y, y2) and torch.equal(y, y3)
    # bf16 outputs are the rounding of the float32 ones
    layer.lin.y_dtype = L.QE_BF16
    assert torch.equal(layer.forward(x.to(DEV)), y.to(torch.bfloat16))


def test_steps_equal_the_forward(Q):
    """qe_route + qe_adapter_inputs + qe_mx4_quant + qe_mx4_gemm give the forward's result.  The forward takes
    the routes, u and v from one pass and qe_adapter_inputs u and v from another, whose K splits may differ: the
    float32 sums behind u and v then differ by rounding, so an entry of u or v can round to the other bf16
    neighbour, one step (at most 2^-7 of it) away.  Hence |dy| <= 2^-7 (|u| |B_s| + |v| |B_e|), plus the
    float32 sums' own n 2^-23 sum|terms| on either side."""
    L = Q.libqe
    cfg = synth.get_config("qwen2vl_2b")
    spec = next(l for l in cfg.linears if l.name == "k")
    params = synth.gen_linear(cfg, spec)
    layer = Q.QELinear.from_params(params, 4, 4, device=DEV)
    s = _dev(params["s"])
    for T in (5, 300):
        x = synth.gen_activations(cfg, spec.stream, T=T).to(DEV)
        e_f = torch.empty(T, dtype=torch.int32, device=DEV)
        y_f = layer.forward(x, expert_out=e_f)
        ws = layer.workspace(T)
        i32 = lambda *n: torch.empty(*n, dtype=torch.int32, device=DEV)  # noqa: E731
        e, counts, offsets, perm = i32(T), i32(8), i32(9), i32(T)
        L.qe_route(layer.lin, x, None, e, counts, offsets, perm, ws)
        u = torch.empty(T, 32, dtype=torch.bfloat16, device=DEV)
        v = torch.empty_like(u)
        L.qe_adapter_inputs(layer.lin, x, e, u, v, ws)
        codes = torch.empty(T, spec.d_in // 2, dtype=torch.uint8, device=DEV)
        scales = torch.empty(T, spec.d_in // 32, dtype=torch.uint8, device=DEV)
        L.qe_mx4_quant(x, s, codes, scales)
        y = torch.empty_like(y_f)
        L.qe_mx4_gemm(layer.lin, codes, scales, u, v, e, y, ws, perm=perm)
        assert torch.equal(e, e_f)
        a, w = (M.mx4_values(M.unpack(c.cpu().numpy()), t.cpu().numpy())
                for c, t in ((codes, scales), (layer.packed, layer.w_scale)))
        B_s, B_r, u, v, e = (t.double().cpu().numpy() for t in (params["B_s"], params["B_r"], u, v, e))
        _, mag = M.mx4_gemm(a, w, u, B_s, v, e, B_r)
        _, adapters = M.mx4_gemm(a * 0, w, u, B_s, v, e, B_r)
        tol = 2.0 ** -7 * adapters + 2 * (spec.d_in + 64) * 2.0 ** -23 * mag
        assert np.all(np.abs((y.double() - y_f.double()).cpu().numpy()) <= tol)


def test_top2_forward(Q):
    """Both routed corrections: the forward plus the second expert's term, added in float32."""
    L = Q.libqe
    cfg = synth.get_config("tiny")
    spec = cfg.linears[0]
    params = synth.gen_linear(cfg, spec)
    layer = Q.QELinear.from_params(params, 4, 4, device=DEV)
    x = synth.gen_activations(cfg, spec.stream)
    T = x.shape[0]
    y1 = layer.forward(x.to(DEV))
    e1, e2 = (torch.empty(T, dtype=torch.int32, device=DEV) for _ in range(2))
    y2 = torch.empty_like(y1)
    ws = torch.empty(L.qe_top2_workspace_bytes(layer.lin, T), dtype=torch.uint8, device=DEV)
    L.qe_linear_forward_top2(layer.lin, x.to(DEV), y2, e1, e2, ws)
    assert bool((e1 != e2).all())
    xb = x.to(torch.bfloat16).double().numpy()
    e2 = e2.cpu().numpy()
    v = np.stack([xb[t] @ params["A_r"][e2[t]].double().numpy() for t in range(T)])
    B = params["B_r"].double().numpy()
    term = np.stack([v[t] @ B[e2[t]] for t in range(T)])
    mag = np.stack([np.abs(v[t]) @ np.abs(B[e2[t]]) for t in range(T)])
    got = (y2.double() - y1.double()).cpu().numpy()
    # v in bf16 (2^-8), float32 sums of 256 and 8 terms, and the sum with y rounded to float32
    vm = np.stack([np.abs(xb[t]) @ np.abs(params["A_r"][e2[t]].double().numpy()) for t in range(T)])
    slack = np.stack([vm[t] @ np.abs(B[e2[t]]) for t in range(T)])
    tol = 2.0 ** -8 * mag + 300 * 2.0 ** -23 * (slack + np.abs(y2.double().cpu().numpy()))
    assert np.all(np.abs(got - term) <= tol)


@pytest.mark.parametrize("T", [1, 40, 700])
def test_group_of_mixed_linears(Q, T):
    """A group forward is its linears' own forwards, whatever their settings."""
    L = Q.libqe
    cfg = synth.get_config("qwen2vl_2b")
    specs = {l.name: l for l in cfg.linears}
    x = synth.gen_activations(cfg, specs["q"].stream, T=T).to(DEV)
    layers = [Q.QELinear.from_params(synth.gen_linear(cfg, specs[n]), 4, a, device=DEV)
              for n, a in (("q", 4), ("k", 8), ("v", 4))]
    own_e = [torch.full((T,), -1, dtype=torch.int32, device=DEV) for _ in layers]
    own = [l.forward(x, expert_out=e) for l, e in zip(layers, own_e)]
    for pick in ([0, 1, 2], [0, 2], [2]):
        y = [torch.empty_like(own[i]) for i in pick]
        e = [torch.empty_like(own_e[i]) for i in pick]
        L.qe_group_forward([layers[i].lin for i in pick], x, y, e, [layers[i].workspace(T) for i in pick])
        for i, a, b in zip(pick, y, e):
            assert torch.equal(a, own[i]) and torch.equal(b, own_e[i])


@pytest.mark.parametrize("T", [9, 300])
def test_routed_term_added_apart(Q, T):
    """qe_mx4_gemm without the routed term, then qe_routed_lora, which adds (bf16(x) . A_e) . B_e: v is rounded to
    bf16 in both ways from float32 sums that may differ, so |dy| <= 2^-7 |v| |B_e| plus float32 rounding."""
    L = Q.libqe
    cfg = synth.get_config("qwen2vl_2b")
    spec = next(l for l in cfg.linears if l.name == "k")
    params = synth.gen_linear(cfg, spec)
    layer = Q.QELinear.from_params(params, 4, 4, device=DEV)
    x = synth.gen_activations(cfg, spec.stream, T=T).to(DEV)
    ws = layer.workspace(T)
    i32 = lambda n: torch.empty(n, dtype=torch.int32, device=DEV)  # noqa: E731
    e, counts, offsets, perm = i32(T), i32(cfg.n_routed), i32(cfg.n_routed + 1), i32(T)
    L.qe_route(layer.lin, x, None, e, counts, offsets, perm, ws)
    u = torch.empty(T, L.rank_pad(cfg.r_shared), dtype=torch.bfloat16, device=DEV)
    v = torch.empty(T, L.rank_pad(cfg.r_routed), dtype=torch.bfloat16, device=DEV)
    L.qe_adapter_inputs(layer.lin, x, e, u, v, ws)
    codes = torch.empty(T, spec.d_in // 2, dtype=torch.uint8, device=DEV)
    scales = torch.empty(T, spec.d_in // 32, dtype=torch.uint8, device=DEV)
    L.qe_mx4_quant(x, _dev(params["s"]), codes, scales)
    y = [torch.empty(T, spec.d_out, dtype=torch.float32, device=DEV) for _ in range(2)]
    L.qe_mx4_gemm(layer.lin, codes, scales, u, v, e, y[0], ws)
    L.qe_mx4_gemm(layer.lin, codes, scales, u, None, None, y[1], ws)
    L.qe_routed_lora(layer.lin, x, e, offsets, perm, y[1], ws)
    a, w = (M.mx4_values(M.unpack(c.cpu().numpy()), t.cpu().numpy())
            for c, t in ((codes, scales), (layer.packed, layer.w_scale)))
    B_s, B_r, u, v, e = (t.double().cpu().numpy() for t in (params["B_s"], params["B_r"], u, v, e))
    u, v, e = u[:, :cfg.r_shared], v[:, :cfg.r_routed], e.astype(np.int32)
    _, mag = M.mx4_gemm(a, w, u, B_s, v, e, B_r)
    _, routed = M.mx4_gemm(a * 0, w, None, None, v, e, B_r)
    tol = 2.0 ** -7 * routed + 2 * (spec.d_in + 64) * 2.0 ** -23 * mag
    assert np.all(np.abs((y[0].double() - y[1].double()).cpu().numpy()) <= tol)


def test_no_tokens(Q):
    """Calls without tokens return at once and leave everything as it was."""
    L = Q.libqe
    rng = np.random.default_rng(2)
    layer = Q.QELinear.from_params(dict(W_f=rng.standard_normal((48, 256)).astype(np.float32)), 4, 4, device=DEV)
    u8 = lambda n: torch.empty(0, n, dtype=torch.uint8, device=DEV)  # noqa: E731
    x = torch.empty(0, 256, dtype=torch.bfloat16, device=DEV)
    w = torch.ones(256, device=DEV)
    ws = torch.empty(256, dtype=torch.uint8, device=DEV)
    y = torch.empty(0, 48, device=DEV)
    L.qe_mx4_quant(x, w, u8(128), u8(8))
    L.qe_mx4_dequant(u8(128), u8(8), x)
    L.qe_mx4_gemm(layer.lin, u8(128), u8(8), None, None, None, y, ws)
    L.qe_add_rmsnorm(x, x, w, 1e-6, h=x.clone(), xn=x.clone(), a_bits=4, codes=u8(128), scales=u8(8))
    L.qe_linear_forward(layer.lin, x, y, None, ws)
    torch.cuda.synchronize()
