"""The microscaled operators as a decoder layer uses them: residual addition and norm with codes, the
products of the linears that read them, and the next norm; in one stream, captured in a HIP graph and
replayed, on two streams at once, and for one token.

The chain's result is compared with the float64 oracle of every step on the step's own inputs, so that a
rounding of one step does not hide an error of the next.
"""

import numpy as np
import pytest
import torch

import synth
from oracle import qe_mx4_oracle as M

pytestmark = pytest.mark.gpu
DEV = "cuda"
D, KV, FF = 512, 256, 1408  # model, key and feed-forward widths


@pytest.fixture(scope="module")
def Q():
    import quantized_linear_moe_amd as q
    return q


def _params(rng, d_in, d_out, s):
    bf = lambda *shape: torch.from_numpy((0.02 * rng.standard_normal(shape)).astype(np.float32)).to(torch.bfloat16)  # noqa: E731
    return dict(W_f=(0.02 * rng.standard_normal((d_out, d_in))).astype(np.float32), s=s, A_s=bf(d_in, 16), B_s=bf(16, d_out),
                A_r=bf(4, d_in, 8), B_r=bf(4, 8, d_out), R=bf(d_in, 4))


class Layer:
    """Norm, then three linears on its codes, and a norm of their sum's residual: q and k read the first norm,
    `o` is fed with q's output."""

    def __init__(self, Q, seed=0):
        rng = np.random.default_rng(seed)
        self.L = Q.libqe
        self.s = rng.uniform(0.5, 2.0, D).astype(np.float32)
        self.p = {n: _params(rng, D, o, self.s) for n, o in (("q", D), ("k", KV), ("up", FF))}
        self.lin = {n: Q.QELinear.from_params(p, 4, 4, device=DEV) for n, p in self.p.items()}
        self.lin["q"].lin.y_dtype = self.L.QE_BF16
        t = lambda a: torch.from_numpy(a).to(DEV)  # noqa: E731
        self.smooth = t(self.s)
        self.w = [t((1 + 0.1 * rng.standard_normal(D)).astype(np.float32)).to(torch.bfloat16) for _ in range(2)]

    def buffers(self, T):
        e = lambda *shape, dtype=torch.bfloat16: torch.empty(*shape, dtype=dtype, device=DEV)  # noqa: E731
        i32, u8 = torch.int32, torch.uint8
        b = dict(h=e(T, D), xn=e(T, D), codes=e(T, D // 2, dtype=u8), scales=e(T, D // 32, dtype=u8), h2=e(T, D), xn2=e(T, D),
                 codes2=e(T, D // 2, dtype=u8), scales2=e(T, D // 32, dtype=u8))
        for n, l in self.lin.items():
            b[n] = dict(y=e(T, l.lin.d_out, dtype=torch.bfloat16 if n == "q" else torch.float32), expert=e(T, dtype=i32),
                        counts=e(4, dtype=i32), offsets=e(5, dtype=i32), perm=e(T, dtype=i32), u=e(T, 32), v=e(T, 32),
                        ws=l.workspace(T))
        return b

    def run(self, x, res, b):
        L = self.L
        L.qe_add_rmsnorm(x, res, self.w[0], 1e-6, h=b["h"], xn=b["xn"], smooth=self.smooth, a_bits=4, codes=b["codes"],
                         scales=b["scales"])
        for n in ("q", "k"):
            self.product(n, b["xn"], b["codes"], b["scales"], b[n])
        L.qe_add_rmsnorm(b["q"]["y"], b["h"], self.w[1], 1e-6, h=b["h2"], xn=b["xn2"], smooth=self.smooth, a_bits=4,
                         codes=b["codes2"], scales=b["scales2"])
        self.product("up", b["xn2"], b["codes2"], b["scales2"], b["up"])

    def product(self, n, xn, codes, scales, c):
        L, lin = self.L, self.lin[n].lin
        L.qe_route(lin, xn, None, c["expert"], c["counts"], c["offsets"], c["perm"], c["ws"])
        L.qe_adapter_inputs(lin, xn, c["expert"], c["u"], c["v"], c["ws"])
        L.qe_mx4_gemm(lin, codes, scales, c["u"], c["v"], c["expert"], c["y"], c["ws"], perm=c["perm"])

    def outputs(self, b):
        return [b[k] for k in ("h", "xn", "codes", "scales", "h2", "xn2", "codes2", "scales2")] + \
            [b[n][k] for n in self.lin for k in ("y", "expert", "u", "v")]


def _inputs(T, seed):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(T, D, generator=g)
    x[:, 5] *= 30
    return x.to(torch.bfloat16).to(DEV), torch.randn(T, D, generator=g).to(torch.bfloat16).to(DEV)


def _f(t):
    return t.float().cpu().numpy()


def _check_norm(x, res, w, s, h, xn, codes, scales):
    ref_h, ref_xn = M.add_rmsnorm(_f(x), _f(res), _f(w), 1e-6, True)
    assert np.array_equal(_f(h), ref_h) and np.array_equal(_f(xn), ref_xn)
    ref_c, ref_s = M.mx4_quant(M.smooth(ref_xn, s, False))
    c = M.unpack(codes.cpu().numpy())
    assert np.array_equal(scales.cpu().numpy(), ref_s)
    assert np.array_equal(np.where((c & 7) == 0, 0, c), np.where((ref_c & 7) == 0, 0, ref_c))


def _check_product(p, codes, scales, c, y):
    a = M.mx4_values(M.unpack(codes.cpu().numpy()), scales.cpu().numpy())
    w = M.mx4_values(*M.mx4_quant(M.smooth(p["W_f"], p["s"], True)))
    e = c["expert"].cpu().numpy()
    ref, mag = M.mx4_gemm(a, w, _f(c["u"])[:, :16], p["B_s"].double().numpy(), _f(c["v"])[:, :8], e, p["B_r"].double().numpy())
    tol = (D + 24) * 2.0 ** -23 * mag + (2.0 ** -8 * np.abs(ref) * (1 + 2.0 ** -8) if y.dtype == torch.bfloat16 else 0)
    assert np.all(np.abs(_f(y).astype(np.float64) - ref) <= tol)


@pytest.mark.parametrize("T", [1, 3, 16, 65, 300, 1500])
def test_chain(Q, T):
    layer = Layer(Q)
    x, res = _inputs(T, T)
    b = layer.buffers(T)
    layer.run(x, res, b)
    torch.cuda.synchronize()
    _check_norm(x, res, layer.w[0], layer.s, b["h"], b["xn"], b["codes"], b["scales"])
    _check_norm(b["q"]["y"], b["h"], layer.w[1], layer.s, b["h2"], b["xn2"], b["codes2"], b["scales2"])
    for n, c, s in (("q", "codes", "scales"), ("k", "codes", "scales"), ("up", "codes2", "scales2")):
        _check_product(layer.p[n], b[c], b[s], b[n], b[n]["y"])


def _poison(outs):
    for o in outs:
        o.fill_(float("nan") if o.is_floating_point() else 99)


@pytest.mark.parametrize("T", [1, 40, 700])
def test_chain_graph_replays(Q, T):
    """Captured once and replayed with the program's own eager work between; two graphs share the workspaces."""
    layer = Layer(Q)
    b = layer.buffers(T)
    ins = [_inputs(T, k) for k in range(2)]
    x, res = ins[0][0].clone(), ins[0][1].clone()
    refs = []
    for xi, ri in ins:
        layer.run(xi, ri, b)
        torch.cuda.synchronize()
        refs.append([o.clone() for o in layer.outputs(b)])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        layer.run(x, res, b)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            layer.run(x, res, b)
        graphs.append(g)
    outs = layer.outputs(b)
    for r in range(4):
        k = r % 2
        x.copy_(ins[k][0])
        res.copy_(ins[k][1])
        _poison(outs)
        graphs[r // 2].replay()
        torch.cuda.synchronize()
        for i, (o, ref) in enumerate(zip(outs, refs[k])):
            assert torch.equal(o.view(torch.uint8), ref.view(torch.uint8)), f"replay {r}, output {i}"
        layer.run(ins[1 - k][0], ins[1 - k][1], b)  # the program's own eager work on the same buffers
        torch.cuda.synchronize()


def test_two_streams_at_once(Q):
    """Two calls in flight on two streams, each with its own workspace and outputs."""
    layer = Layer(Q)
    T = 900
    bufs = [layer.buffers(T) for _ in range(2)]
    ins = [_inputs(T, 10 + k) for k in range(2)]
    refs = []
    for k in range(2):
        layer.run(*ins[k], bufs[k])
        torch.cuda.synchronize()
        refs.append([o.clone() for o in layer.outputs(bufs[k])])
        _poison(layer.outputs(bufs[k]))
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(3):
        for k in range(2):
            with torch.cuda.stream(streams[k]):
                layer.run(*ins[k], bufs[k])
    torch.cuda.synchronize()
    for k in range(2):
        for o, ref in zip(layer.outputs(bufs[k]), refs[k]):
            assert torch.equal(o.view(torch.uint8), ref.view(torch.uint8))


@pytest.mark.parametrize("cfg_name,lin_name,T", [("qwen2vl_2b", "k", 8), ("qwen2vl_2b", "k", 100), ("qwen2vl_2b", "gate", 1200), ("qwen2vl_2b", "gate", 1900)])
def test_linear_forward_graph_replays(Q, cfg_name, lin_name, T):
    L = Q.libqe
    cfg = synth.get_config(cfg_name)
    spec = next(l for l in cfg.linears if l.name == lin_name)
    layer = Q.QELinear.from_params(synth.gen_linear(cfg, spec), 4, 4, device=DEV)
    x = synth.gen_activations(cfg, spec.stream, T=T).to(DEV)
    x2 = x.flip(0).contiguous()
    ws = layer.workspace(T)
    y, y2 = (torch.empty(T, spec.d_out, dtype=torch.float32, device=DEV) for _ in range(2))
    e = torch.empty(T, dtype=torch.int32, device=DEV)
    L.qe_linear_forward(layer.lin, x, y, e, ws)
    torch.cuda.synchronize()
    ref, ref_e = y.clone(), e.clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        L.qe_linear_forward(layer.lin, x, y, e, ws)
    for r in range(4):
        y.fill_(float("nan"))
        e.fill_(-5)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, ref) and torch.equal(e, ref_e), f"replay {r}"
        L.qe_linear_forward(layer.lin, x2, y2, e, ws)  # other inputs through the same workspace
        torch.cuda.synchronize()


def test_given_stream_is_used(Q):
    """The stream argument: work is ordered on it and not on the current stream."""
    L = Q.libqe
    side = torch.cuda.Stream()
    x, res = _inputs(64, 3)
    w = torch.ones(D, dtype=torch.bfloat16, device=DEV)
    h, xn = torch.empty_like(x), torch.empty_like(x)
    codes = torch.empty(64, D // 2, dtype=torch.uint8, device=DEV)
    scales = torch.empty(64, D // 32, dtype=torch.uint8, device=DEV)
    back = torch.empty_like(x)
    torch.cuda.synchronize()
    L.qe_add_rmsnorm(x, res, w, 1e-6, h=h, xn=xn, a_bits=4, codes=codes, scales=scales, stream=side)
    L.qe_mx4_dequant(codes, scales, back, stream=side)
    side.synchronize()
    ref_h, ref_xn = M.add_rmsnorm(_f(x), _f(res), _f(w), 1e-6, True)
    assert np.array_equal(_f(xn), ref_xn)
    assert np.array_equal(_f(back), M.mx4_values(*M.mx4_quant(ref_xn)).astype(np.float32))
