"""Workloads of the operators around the microscaled 4-bit linear: the residual addition with RMS
norm and quantized output, the microscaled quantization, and the product of two microscaled operands
with the low-rank corrections.

With `own` False, run() computes an operator in elementary torch operations; with `own` True it calls
the library's entry points.  A case is a dict of plain values; "op" names the operator:

  norm   T tokens of d channels, type x; h = x + res (res False: h = x), xn = RMS norm of h, and xn as
         a_bits 4 (microscaled blocks), 6 or 8 (per-token integer) codes after division by a smoothing
         vector (smooth True).  Outputs: h, xn and the values the codes stand for.
  quant  a [T][d] tensor, divided by ("div", activations) or multiplied with ("mul", weights) a
         smoothing vector, or neither (""), in microscaled blocks, and read back.
  gemm   T tokens, d_in -> d_out, both operands microscaled, y in type y, shared-expert rank r_s,
         n_r routed experts of rank r_r (tokens visited in expert order when perm is True).
"""

import math

import torch

own = False
DEV = "cuda"
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
EPS = 1e-6


def listed():
    return [
        # one token in front of a 2B-sized layer's q/k/v: the call is all latency
        dict(name="norm_T1_d1536_mx4", op="norm", T=1, d=1536, x="bf16", res=True, a_bits=4, smooth=True),
        # prefill of a 2B-sized layer, 6-bit codes for the integer product
        dict(name="norm_T2048_d1536_a6", op="norm", T=2048, d=1536, x="bf16", res=True, a_bits=6, smooth=True),
        # a float32 stream with a ragged token count, its first norm (nothing to add yet), 8-bit codes
        dict(name="norm_T333_d4096_a8_f32", op="norm", T=333, d=4096, x="f32", res=False, a_bits=8, smooth=True),
        # prefill of a 72B-sized layer, microscaled codes
        dict(name="norm_T4096_d8192_mx4", op="norm", T=4096, d=8192, x="bf16", res=True, a_bits=4, smooth=True),
        # decode activations in front of a 72B-sized down projection
        dict(name="quant_T8_d29568_div", op="quant", T=8, d=29568, x="bf16", smooth="div"),
        # prefill activations in front of an 8B-sized down projection, ragged token count
        dict(name="quant_T4093_d14336_div", op="quant", T=4093, d=14336, x="bf16", smooth="div"),
        # load time: one 72B-sized weight matrix with its smoothing factors
        dict(name="quant_72b_weights_mul", op="quant", T=29568, d=8192, x="f32", smooth="mul"),
        # one token through a 72B-sized gate or up projection, no corrections: weight streaming
        dict(name="gemm_T1_8192x29568", op="gemm", T=1, d_in=8192, d_out=29568, y="f32", r_s=0, n_r=0, r_r=0, perm=False),
        # a few decode streams through the 72B-sized down projection with all corrections, bf16 out
        dict(name="gemm_T8_29568x8192_qe", op="gemm", T=8, d_in=29568, d_out=8192, y="bf16", r_s=32, n_r=8, r_r=32,
             perm=False),
        # a short prompt through a 7B-sized up projection
        dict(name="gemm_T128_3584x18944_qe", op="gemm", T=128, d_in=3584, d_out=18944, y="f32", r_s=32, n_r=8, r_r=32,
             perm=False),
        # a ragged prefill through a narrow 2B-sized key projection, odd ranks
        dict(name="gemm_T2041_1536x256_qe", op="gemm", T=2041, d_in=1536, d_out=256, y="bf16", r_s=8, n_r=4, r_r=48,
             perm=True),
        # prefill through a 72B-sized gate or up projection, tokens in expert order
        dict(name="gemm_T4096_8192x29568_qe", op="gemm", T=4096, d_in=8192, d_out=29568, y="f32", r_s=32, n_r=8, r_r=32,
             perm=True),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("norm", "quant", "gemm", "gemm"))
    if op == "norm":
        return dict(op=op, T=_log(rng, 1, 4096), d=32 * _log(rng, 4, 256), x=rng.choice(("bf16", "bf16", "f32")),
                    res=rng.random() < 0.8, a_bits=rng.choice((4, 6, 8)), smooth=rng.random() < 0.7)
    if op == "quant":
        return dict(op=op, T=_log(rng, 1, 29568), d=32 * _log(rng, 4, 256), x=rng.choice(("bf16", "f32")),
                    smooth=rng.choice(("div", "mul", "")))
    n_r = rng.choice((0, 4, 8, 16))
    return dict(op=op, T=_log(rng, 1, 4096), d_in=128 * _log(rng, 2, 64), d_out=16 * _log(rng, 16, 1848),
                y=rng.choice(("f32", "bf16")), r_s=rng.choice((0, 16, 32, 64)), n_r=n_r,
                r_r=rng.choice((8, 32, 64)) if n_r else 0, perm=bool(n_r) and rng.random() < 0.5)


# ------------------------------------------------------------------------ inputs
def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    return g


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device=DEV)


def _activations(g, T, d):
    """Gaussian tokens with a few channels that are large on every token."""
    x = _randn(g, T, d)
    x[:, torch.randint(0, d, (8,), generator=g, device=DEV)] *= 30.0
    return x


def _pad32(r):
    return (r + 31) // 32 * 32


def _rank_rows(g, T, r, d_in):
    """bf16 adapter inputs of T tokens (rows padded with zeros to whole steps of 32)."""
    u = torch.zeros(T, _pad32(r), dtype=torch.bfloat16, device=DEV)
    u[:, :r] = (_randn(g, T, r) * (0.02 * math.sqrt(d_in))).to(torch.bfloat16)
    return u


def prepare(case, seed):
    g = _gen(seed)
    s = dict(case)
    op = case["op"]
    if op == "norm":
        T, d, dt = case["T"], case["d"], DTYPES[case["x"]]
        s["input"] = _activations(g, T, d).to(dt)
        s["residual"] = _activations(g, T, d).to(dt) if case["res"] else None
        s["weight"] = (1.0 + 0.1 * _randn(g, d)).to(dt)
        s["factors"] = 0.5 + 1.5 * torch.rand(d, generator=g, device=DEV) if case["smooth"] else None
    elif op == "quant":
        T, d = case["T"], case["d"]
        x = 0.02 * _randn(g, T, d) if case["smooth"] == "mul" else _activations(g, T, d)
        s["input"] = x.to(DTYPES[case["x"]])
        s["factors"] = 0.5 + 1.5 * torch.rand(d, generator=g, device=DEV) if case["smooth"] else None
    else:
        T, d_in, d_out = case["T"], case["d_in"], case["d_out"]
        s["codes"], s["scales"] = _mx4(_activations(g, T, d_in))
        s["w_codes"], s["w_scales"] = _mx4(0.02 * _randn(g, d_out, d_in))
        if case["r_s"]:
            s["u"] = _rank_rows(g, T, case["r_s"], d_in)
            s["B_s"] = (0.02 * _randn(g, case["r_s"], d_out)).to(torch.bfloat16)
        if case["n_r"]:
            s["v"] = _rank_rows(g, T, case["r_r"], d_in)
            s["B_r"] = (0.02 * _randn(g, case["n_r"], case["r_r"], d_out)).to(torch.bfloat16)
            s["expert"] = torch.randint(0, case["n_r"], (T,), generator=g, device=DEV).to(torch.int32)
            s["order"] = torch.argsort(s["expert"], stable=True).to(torch.int32) if case["perm"] else None
    if own:
        _buffers(s)
    return s


# --------------------------------------------------- what a user's program keeps
def _buffers(s):
    """Output buffers, and for the product the prepared weights and the workspace."""
    from quantized_linear_moe_amd import libqe as L
    op = s["op"]
    empty = lambda *shape, dtype: torch.empty(*shape, dtype=dtype, device=DEV)  # noqa: E731
    if op == "gemm":
        T, d_in, d_out, r_s, n_r, r_r = (s[k] for k in ("T", "d_in", "d_out", "r_s", "n_r", "r_r"))
        lin = L.make_linear(d_in, d_out, 4, 4, r_s, n_r, r_r)
        lin.y_dtype = L.QE_BF16 if s["y"] == "bf16" else L.QE_F32
        s["prep"] = empty(L.qe_prepared_bytes(lin), dtype=torch.uint8)
        lin.prep = s["prep"].data_ptr()
        zeros = lambda *shape: torch.zeros(*shape, dtype=torch.bfloat16, device=DEV)  # noqa: E731
        L.qe_mx4_prepare(lin, s["w_codes"], s["w_scales"], None, zeros(d_in, r_s) if r_s else None, s.get("B_s"),
                         zeros(n_r, d_in, r_r) if n_r else None, s.get("B_r"), zeros(d_in, n_r) if n_r else None,
                         s["prep"])
        torch.cuda.synchronize()
        s["lin"] = lin
        s["ws"] = empty(max(L.qe_workspace_bytes(lin, T), 256), dtype=torch.uint8)
        s["out"] = empty(T, d_out, dtype=DTYPES[s["y"]])
        return
    T, d = s["T"], s["d"]
    s["values"] = empty(T, d, dtype=torch.bfloat16)
    if op == "quant" or s["a_bits"] == 4:
        s["q"], s["q_scales"] = empty(T, d // 2, dtype=torch.uint8), empty(T, d // 32, dtype=torch.uint8)
    else:
        s["q"], s["q_scales"] = empty(T, d, dtype=torch.int8), empty(T, dtype=torch.float32)
    if op == "norm":
        s["h"], s["xn"] = torch.empty_like(s["input"]), torch.empty_like(s["input"])


def _run_own(s):
    from quantized_linear_moe_amd import libqe as L
    op = s["op"]
    if op == "gemm":
        L.qe_mx4_gemm(s["lin"], s["codes"], s["scales"], s.get("u"), s.get("v"), s.get("expert"), s["out"], s["ws"],
                      perm=s.get("order"))
        return {"y": s["out"]}
    if op == "quant":
        L.qe_mx4_quant(s["input"], s["factors"], s["q"], s["q_scales"], multiply=s["smooth"] == "mul")
        L.qe_mx4_dequant(s["q"], s["q_scales"], s["values"])
        return {"values": s["values"]}
    L.qe_add_rmsnorm(s["input"], s["residual"], s["weight"], EPS, h=s["h"], xn=s["xn"], smooth=s["factors"],
                     a_bits=s["a_bits"], codes=s["q"], scales=s["q_scales"])
    if s["a_bits"] == 4:
        L.qe_mx4_dequant(s["q"], s["q_scales"], s["values"])
    else:
        torch.mul(s["q"], s["q_scales"][:, None], out=s["values"])
    return {"h": s["h"], "xn": s["xn"], "values": s["values"]}


# -------------------------------------------------------------------- plain forms
def _mx4_levels(x):
    """The microscaled form of float32 x: level indices 0..7 of |x|, signs, and the exponent field of
    every block's scale (2^(field - 127), two below the field of the block's largest magnitude)."""
    T, d = x.shape
    blocks = x.reshape(T, d // 32, 32)
    bits = blocks.abs().amax(-1).view(torch.int32)
    field = ((bits >> 23) - 2).clamp_(min=0)
    z = (blocks * ((254 - field) << 23).view(torch.float32)[..., None]).abs()
    # nearest level of 0, .5, 1, 1.5, 2, 3, 4, 6; a value halfway takes the even index
    level = (z > 0.25).to(torch.uint8)
    level += z >= 0.75
    level += z > 1.25
    level += z >= 1.75
    level += z > 2.5
    level += z >= 3.5
    level += z > 5.0
    return level, torch.signbit(blocks), field


def _mx4(x):
    """Packed codes [T][d/2] (even channel in the low nibble) and scales [T][d/32]."""
    level, sign, field = _mx4_levels(x)
    code = (level | (sign.to(torch.uint8) << 3)).reshape(x.shape[0], -1, 2)
    return code[..., 0] | (code[..., 1] << 4), field.to(torch.uint8)


def _mx4_values(x):
    """The values the microscaled form of float32 x stands for, float32."""
    level, sign, field = _mx4_levels(x)
    table = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], device=x.device)
    v = table[level.int()] * _exp2(field)[..., None]
    return torch.where(sign, -v, v).reshape(x.shape)


def _exp2(field):
    """2^(field - 127) for exponent fields 0..254, exactly."""
    return ((field.to(torch.int64) + 896) << 52).view(torch.float64).float()


def _unpack(codes, scales):
    """float32 values of packed codes and scales."""
    table = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0],
                         device=codes.device)
    v = torch.stack((table[(codes & 15).int()], table[(codes >> 4).int()]), -1)
    T = codes.shape[0]
    return (v.reshape(T, -1, 32) * _exp2(scales)[..., None]).reshape(T, -1)


def _run_plain(s):
    op = s["op"]
    if op == "gemm":
        y = _unpack(s["codes"], s["scales"]) @ _unpack(s["w_codes"], s["w_scales"]).t()
        if s["r_s"]:
            y += s["u"][:, : s["r_s"]].float() @ s["B_s"].float()
        if s["n_r"]:  # every token's row in its own expert's columns, then one product
            T, r_r, n_r = s["T"], s["r_r"], s["n_r"]
            mine = s["expert"].long()[:, None] == torch.arange(n_r, device=DEV)
            v = s["v"][:, None, :r_r].float() * mine[..., None]
            y += v.reshape(T, n_r * r_r) @ s["B_r"].float().reshape(n_r * r_r, -1)
        return {"y": y.to(DTYPES[s["y"]])}
    x = s["input"].float()
    if op == "quant":
        if s["smooth"]:
            x = x / s["factors"] if s["smooth"] == "div" else x * s["factors"]
        return {"values": _mx4_values(x).to(torch.bfloat16)}
    dt = s["input"].dtype
    h = x if s["residual"] is None else (x + s["residual"].float()).to(dt).float()
    # the mean in 64 bits: codes of values next to a border depend on its last place in 32
    rstd = torch.rsqrt(h.double().square().mean(-1, keepdim=True) + EPS).float()
    xn = ((h * rstd) * s["weight"].float()).to(dt)
    z = xn.float()
    if s["factors"] is not None:
        z = z / s["factors"]
    if s["a_bits"] == 4:
        values = _mx4_values(z)
    else:
        q = 2 ** (s["a_bits"] - 1) - 1
        scale = z.abs().amax(-1, keepdim=True) / q
        values = torch.round(z / scale).clamp_(-q, q) * scale
    return {"h": h.to(dt), "xn": xn, "values": values.to(torch.bfloat16)}


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ------------------------------------------------------------------- work, exact
def work(case):
    op = case["op"]
    if op == "gemm":
        T, d_in, d_out, r_s, n_r, r_r = (case[k] for k in ("T", "d_in", "d_out", "r_s", "n_r", "r_r"))
        b = (T + d_out) * d_in * (1 / 2 + 1 / 32) + T * d_out * (2 if case["y"] == "bf16" else 4)
        b += 2 * (T + d_out) * r_s + (2 * T * r_r + 4 * T + 2 * min(n_r, T) * r_r * d_out if n_r else 0)
        return {"bytes": b, "flops": 2.0 * T * d_out * (d_in + r_s + r_r)}
    n = case["T"] * case["d"]
    e = 2 if case["x"] == "bf16" else 4
    if op == "quant":
        return {"bytes": n * (e + 2) + 4 * case["d"], "flops": 4.0 * n}
    return {"bytes": n * (e * (3 + (1 if case["res"] else 0)) + 2) + case["d"] * (e + 4), "flops": 9.0 * n}


def _exact_blocks(x):
    """Microscaled values of float64 x, from the definition: per block of 32 the scale is 2^(E - 2) with
    2^E the largest power of two not above the block's largest magnitude; every value goes to the
    nearest multiple of the spacing around it, halfway cases to the even multiple, at most 6 scales."""
    T, d = x.shape
    b = x.reshape(T, d // 32, 32)
    _, exponent = torch.frexp(b.abs().amax(-1, keepdim=True))
    scale = torch.pow(2.0, (exponent - 3).clamp(min=-127).double())
    r = (b / scale).abs()
    spacing = torch.where(r < 2, 0.5, torch.where(r < 4, 1.0, 2.0)).double()
    r = (torch.round(r / spacing) * spacing).clamp_(max=6.0)
    return (torch.copysign(r, b) * scale).reshape(T, d)


def _exact_operand(codes, scales):
    """float64 values of packed codes and scales, by sign, exponent and mantissa bit of every code."""
    T = codes.shape[0]
    c = torch.stack((codes % 16, codes // 16), -1).reshape(T, -1).long()
    exponent, mantissa = (c % 8) // 2, (c % 2).double()
    v = torch.where(exponent > 0, (1 + mantissa / 2) * torch.pow(2.0, (exponent - 1).double()), mantissa / 2)
    v = torch.where(c >= 8, -v, v)
    return v * torch.pow(2.0, scales.double() - 127).repeat_interleave(32, 1)


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "gemm":
        y = _exact_operand(s["codes"], s["scales"]) @ _exact_operand(s["w_codes"], s["w_scales"]).t()
        if case["r_s"]:
            y += s["u"][:, : case["r_s"]].double() @ s["B_s"].double()
        for e in range(case["n_r"]):
            at = (s["expert"] == e).nonzero()[:, 0]
            y[at] += s["v"][at, : case["r_r"]].double() @ s["B_r"][e].double()
        return {"y": y}
    x = s["input"].double()
    f = None if s["factors"] is None else s["factors"].double()
    if op == "quant":
        if case["smooth"]:  # the smoothed value is held in 32 bits
            x = (x / f if case["smooth"] == "div" else x * f).float().double()
        return {"values": _exact_blocks(x)}
    dt = s["input"].dtype
    h = x if s["residual"] is None else (x + s["residual"].double()).to(dt).double()
    w = s["weight"].double()
    xn = h * w / torch.sqrt((h * h).sum(-1, keepdim=True) / case["d"] + EPS)
    z = xn.to(dt).double()
    if f is not None:
        z = (z / f).float().double()
    if case["a_bits"] == 4:
        values = _exact_blocks(z)
    else:
        q = 2 ** (case["a_bits"] - 1) - 1
        scale = z.abs().amax(-1, keepdim=True) / q
        values = torch.round(z / scale).clamp(-q, q) * scale
    return {"h": h, "xn": xn, "values": values}
