"""Workloads of the operators between the quantized linears of a decoding step: rotary positions, keys and values
appended to a paged cache, attention of the new tokens over it, and the verification of drafted tokens.

With `own` False, run() computes an operator in elementary torch operations; with `own` True it calls the
library's entry points.  A case is a dict of plain values; "op" names the operator:

  rope    T tokens of `heads` heads of hd channels, type x, the first rot channels rotated (layout "half": channel
          i with i + rot/2; "pairs": 2i with 2i + 1); sections: how many pairs take each of three rows of positions
          (image tokens), or "" for one row; far: positions start there (long contexts, frequencies scaled for
          them).  Output: y.
  append  T tokens' keys and values (kv heads of hd channels, type x) to a cache of pages, the keys rotated, as
          bf16 or 8-bit codes ("i8", one scale per token and head); q heads rotated on the way (heads 0: none); every
          skip-th token is padding without a place.  Outputs: the values both caches stand for, the rotated q.
  attn    seqs sequences, kv heads of hd channels in a paged cache of that type, heads query heads; new: the
          largest count of new tokens of a sequence, kv: the largest count of keys; ragged: both vary; tree: the new
          tokens are a tree of drafts, else a piece of text.  Output: the attention's rows.
  verify  seqs sequences of up to rows rows (the last accepted token and its drafts), vocab probabilities each; tree:
          chosen tokens with several per parent, else a chain drawn from the drafts' probabilities.
          Outputs: drafts taken, their rows, the token drawn after them.
"""

import math
import random

import numpy as np
import torch

own = False
DEV = "cuda"
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


def listed():
    return [
        # one decoded token of a 2B-sized layer: latency
        dict(name="rope_T1_h12", op="rope", T=1, heads=12, hd=128, rot=128, x="bf16", layout="half", sections="", far=0),
        # part of the head, interleaved, a float32 stream far into a long context
        dict(name="rope_T1000_h32_part_f32", op="rope", T=1000, heads=32, hd=128, rot=64, x="f32", layout="pairs",
             sections="", far=900000),
        # prefill of a 72B-sized layer, image and text tokens, ragged token count
        dict(name="rope_T4093_h64_sections", op="rope", T=4093, heads=64, hd=128, rot=128, x="bf16", layout="half",
             sections="16+24+24", far=0),
        # one decoded token of a 2B-sized layer behind float32 linears
        dict(name="append_T1_h12_kv2", op="append", T=1, heads=12, kv=2, hd=128, rot=128, x="f32", layout="half",
             sections="", far=0, cache="bf16", page=16, skip=0),
        # a ragged batch of an 8B-sized layer with padded places, 8-bit cache
        dict(name="append_T777_h32_kv8_i8", op="append", T=777, heads=32, kv=8, hd=128, rot=128, x="f32",
             layout="half", sections="", far=30000, cache="i8", page=32, skip=9),
        # prefill of a 72B-sized layer
        dict(name="append_T4096_h64_kv8", op="append", T=4096, heads=64, kv=8, hd=128, rot=128, x="bf16",
             layout="half", sections="16+24+24", far=0, cache="bf16", page=16, skip=0),
        # one decoded token of a 2B-sized layer, a short context: latency
        dict(name="attn_1x1_kv1000_h12", op="attn", seqs=1, new=1, kv=1000, heads=12, kv_heads=2, hd=128, cache="bf16",
             page=16, ragged=False, tree=False),
        # a batch decoding a token each through a 72B-sized layer, ragged contexts
        dict(name="attn_64x1_kv8192_h64", op="attn", seqs=64, new=1, kv=8192, heads=64, kv_heads=8, hd=128,
             cache="bf16", page=16, ragged=True, tree=False),
        # trees of drafted tokens through a 7B-sized layer, 8-bit cache
        dict(name="attn_8x48_tree_kv4000_h28_i8", op="attn", seqs=8, new=48, kv=4000, heads=28, kv_heads=4, hd=128,
             cache="i8", page=64, ragged=True, tree=True),
        # a whole prompt through a 72B-sized layer
        dict(name="attn_1x4096_h64", op="attn", seqs=1, new=4096, kv=4096, heads=64, kv_heads=8, hd=128, cache="bf16",
             page=16, ragged=False, tree=False),
        # one stream's chain of drafts
        dict(name="verify_1x5_v32000", op="verify", seqs=1, rows=5, vocab=32000, tree=False),
        # a batch's trees over a large vocabulary
        dict(name="verify_32x33_v131072", op="verify", seqs=32, rows=33, vocab=131072, tree=True),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("rope", "append", "attn", "attn", "verify"))
    if op in ("rope", "append"):
        hd = rng.choice((64, 80, 96, 128, 256))
        rot = min(hd, 16 * rng.randint(1, hd // 16)) if rng.random() < 0.3 else hd
        cut = sorted(rng.randint(0, rot // 2) for _ in range(2))
        c = dict(op=op, T=_log(rng, 1, 4096), hd=hd, rot=rot, x=rng.choice(("bf16", "f32")),
                 layout=rng.choice(("half", "half", "pairs")),
                 sections="%d+%d+%d" % (cut[0], cut[1] - cut[0], rot // 2 - cut[1]) if rng.random() < 0.4 else "",
                 far=rng.choice((0, 1000, 100000, 900000)))
        if op == "rope":
            c.update(heads=_log(rng, 1, 64))
        else:
            kv = rng.choice((1, 2, 4, 8))
            c.update(kv=kv, heads=kv * rng.choice((0, 1, 4, 6, 7, 8)), cache=rng.choice(("bf16", "i8")),
                     page=rng.choice((8, 16, 32, 64, 128)), skip=rng.choice((0, 0, 5)))
        return c
    if op == "verify":
        return dict(op=op, seqs=_log(rng, 1, 32), rows=rng.randint(1, 33), vocab=_log(rng, 1000, 131072),
                    tree=rng.random() < 0.5)
    kind = rng.choice(("token", "tree", "text"))
    kv_heads, group = rng.choice((1, 2, 4, 8)), rng.choice((1, 4, 6, 7, 8))
    c = dict(op=op, heads=kv_heads * group, kv_heads=kv_heads, hd=rng.choice((64, 128, 128)),
             cache=rng.choice(("bf16", "bf16", "i8")), page=rng.choice((8, 16, 32, 64, 128)), ragged=rng.random() < 0.7,
             tree=kind == "tree")
    if kind == "token":
        c.update(seqs=_log(rng, 1, 64), new=1, kv=_log(rng, 1, 8192))
    elif kind == "tree":
        c.update(seqs=_log(rng, 1, 8), new=_log(rng, 2, 100), kv=_log(rng, 128, 8192))
    else:
        c.update(seqs=rng.randint(1, 2), new=_log(rng, 2, 1024))
        c.update(kv=_log(rng, c["new"], 4096))
    return c


# ------------------------------------------------------------------------ inputs
def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    return g


def _sections(case):
    return tuple(int(n) for n in case["sections"].split("+")) if case["sections"] else ()


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device=DEV)


def _heads(g, T, heads, hd):
    """Gaussian heads with one channel of each that is large on every token."""
    x = _randn(g, T, heads, hd)
    x[:, torch.arange(heads, device=DEV), torch.randint(0, hd, (heads,), generator=g, device=DEV)] *= 8.0
    return x


def _rotation(case, g, s):
    """Inverse frequencies (base 1e6; scaled by 1/4 for far positions) and the tokens' positions."""
    rot, T = case["rot"], case["T"]
    f = torch.pow(1e6, -torch.arange(0, rot, 2, dtype=torch.float64, device=DEV) / rot)
    s["inv_freq"] = f / 4 if case["far"] else f
    s["scale"] = 1.0 + 0.1 * math.log(4.0) if case["far"] else 1.0
    text = torch.arange(T, device=DEV)
    if case["sections"]:  # the first three quarters are rows of an image of 40 columns, the rest text
        image = 3 * T // 4
        col, row = text % 40, text // 40
        after = 40 + image // 40 + text - image
        pos = torch.stack((torch.where(text < image, 0, after), torch.where(text < image, row, after),
                           torch.where(text < image, col, after)))
    else:
        pos = text[None]
    s["pos"] = (pos + case["far"]).to(torch.int32).contiguous()


def _lengths(case):
    """New tokens and keys of every sequence of an attention case, or rows of every sequence of a verification."""
    rng = random.Random(case["seqs"] * 1000 + case.get("new", case.get("rows")))
    if case["op"] == "verify":
        return [case["rows"] if b == 0 else rng.randint(1, case["rows"]) for b in range(case["seqs"])]
    new, kv = [], []
    for b in range(case["seqs"]):
        full = b == 0 or not case["ragged"]
        new.append(case["new"] if full else rng.randint(1, case["new"]))
        kv.append(max(new[-1], case["kv"] if full else rng.randint(max(1, case["kv"] // 16), case["kv"])))
    return new, kv


def _draft_tree(rng, n):
    """Parents of n drafted tokens, local: the first hangs on the text (-1), every other on an earlier one."""
    return [-1] + [rng.randint(max(-1, i - 8), i - 1) for i in range(1, n)]


def _prepare_attn(case, seed, g, s):
    rng = random.Random(seed)
    B, hd, kvh, page = case["seqs"], case["hd"], case["kv_heads"], case["page"]
    new, kv = _lengths(case)
    T = sum(new)
    need = [(k + page - 1) // page for k in kv]
    width, pool = max(need), sum(need) + 2
    order = torch.randperm(pool, generator=g, device=DEV).to(torch.int32)
    s["pages"] = torch.zeros(B, width, dtype=torch.int32, device=DEV)
    at = 0
    for b in range(B):
        s["pages"][b, : need[b]] = order[at : at + need[b]]
        at += need[b]
    for name in ("k", "v"):
        x = torch.empty(pool, kvh, page, hd, dtype=torch.bfloat16 if case["cache"] == "bf16" else torch.int8, device=DEV)
        if case["cache"] == "bf16":
            x.normal_(generator=g)
        else:
            x.random_(-127, 128, generator=g)
            s[name + "_scale"] = (0.5 + torch.rand(pool, kvh, page, generator=g, device=DEV)) / 64
        s[name] = x
    s["q"] = (1.5 * _randn(g, T, case["heads"], hd)).to(torch.bfloat16)
    s["new"], s["kv_lens"], s["T"] = new, kv, T
    s["q_start"] = torch.tensor(np.cumsum([0] + new), dtype=torch.int32, device=DEV)
    s["kv_len"] = torch.tensor(kv, dtype=torch.int32, device=DEV)
    s["tree_bits"] = None
    if case["tree"]:  # bit j of a token's row: it sees the j-th new token of its sequence
        words = (max(new) + 31) // 32
        bits = np.zeros((T, words), np.uint32)
        t = 0
        for n in new:
            for i, p in enumerate(_draft_tree(rng, n)):
                if p >= 0:
                    bits[t + i] = bits[t + p]
                bits[t + i, i // 32] |= np.uint32(1 << (i % 32))
            t += n
        s["tree_bits"] = torch.from_numpy(bits.view(np.int32)).to(DEV)


def _prepare_verify(case, seed, g, s):
    rng = random.Random(seed)
    V, B = case["vocab"], case["seqs"]
    rows = _lengths(case)
    N = sum(rows)
    p = torch.empty(N, V, device=DEV)
    p.normal_(0, 3.0, generator=g)
    q = None
    if not case["tree"]:  # the drafts' distributions: the target's logits with noise
        q = torch.empty(N, V, device=DEV)
        q.normal_(generator=g)
        at = 0
        for n in rows:
            q[at + 1 : at + n] += p[at : at + n - 1]
            at += n
        q = torch.softmax(q, -1)
    p = torch.softmax(p, -1)
    parent, drawn_at = [], []
    at = 0
    for n in rows:
        par = [-1] + ([rng.randint(max(0, i - 6), i - 1) for i in range(1, n)] if case["tree"] else list(range(n - 1)))
        parent += par
        drawn_at += [at + max(x, 0) for x in par]
        at += n
    if case["tree"]:  # the most probable tokens of the parent's row, each to one child
        best = torch.topk(p, min(8, V), dim=-1).indices.tolist()
        used, token = {}, []
        for i in range(N):
            k = used.get(drawn_at[i], 0)
            used[drawn_at[i]] = k + (parent[i] >= 0)
            token.append(best[drawn_at[i]][min(k, len(best[0]) - 1)])
        s["token"] = torch.tensor(token, dtype=torch.int32, device=DEV)
    else:
        s["token"] = torch.multinomial(q, 1, generator=g)[:, 0].to(torch.int32)
    s["p"], s["draft_p"], s["rows_of"], s["N"] = p, q, rows, N
    s["parent"] = torch.tensor(parent, dtype=torch.int32, device=DEV) if case["tree"] else None
    s["parents"] = parent
    s["row_start"] = torch.tensor(np.cumsum([0] + rows), dtype=torch.int32, device=DEV)
    s["u"] = torch.rand(N, generator=g, device=DEV)


def prepare(case, seed):
    g = _gen(seed)
    s = dict(case)
    op = case["op"]
    if op == "attn":
        _prepare_attn(case, seed, g, s)
    elif op == "verify":
        _prepare_verify(case, seed, g, s)
    else:
        T, hd, dt = case["T"], case["hd"], DTYPES[case["x"]]
        _rotation(case, g, s)
        if op == "rope":
            s["input"] = _heads(g, T, case["heads"], hd).to(dt)
        else:
            s["k_in"], s["v_in"] = _heads(g, T, case["kv"], hd).to(dt), _heads(g, T, case["kv"], hd).to(dt)
            s["q_in"] = _heads(g, T, case["heads"], hd).to(dt) if case["heads"] else None
            page = case["page"]
            pool = (T + page - 1) // page + 2
            slot = torch.randperm(pool, generator=g, device=DEV)[torch.arange(T, device=DEV) // page] * page
            slot = slot + torch.arange(T, device=DEV) % page
            if case["skip"]:
                slot[:: case["skip"]] = -1
            s["slot"] = slot.to(torch.int32)
            shape = (pool, case["kv"], page, hd)
            for name in ("k", "v"):  # what earlier tokens left
                if case["cache"] == "bf16":
                    s[name] = _randn(g, *shape).to(torch.bfloat16)
                else:
                    s[name] = torch.randint(-127, 128, shape, generator=g, device=DEV).to(torch.int8)
                    s[name + "_scale"] = torch.rand(shape[:3], generator=g, device=DEV) / 64
    if own:
        _buffers(s)
    return s


# --------------------------------------------------- what a user's program keeps
def _buffers(s):
    """Handles, output buffers and workspaces."""
    from quantized_linear_moe_amd import libqe as L
    op = s["op"]
    empty = lambda *shape, dtype: torch.empty(*shape, dtype=dtype, device=DEV)  # noqa: E731
    if op in ("rope", "append"):
        s["rope"] = L.make_rope(s["inv_freq"], pairs=s["layout"] == "pairs", sections=_sections(s) or None,
                                scale=s["scale"])
    if op == "rope":
        s["out"] = torch.empty_like(s["input"])
    if op in ("append", "attn"):
        s["cache_handle"] = L.make_cache(s["k"], s["v"], s.get("k_scale"), s.get("v_scale"))
    if op == "append":
        s["q_out"] = empty(s["T"], s["heads"], s["hd"], dtype=torch.bfloat16) if s["heads"] else None
        if s["cache"] == "i8":
            s["values"] = [empty(*s["k"].shape, dtype=torch.bfloat16) for _ in range(2)]
    if op == "attn":
        s["out"] = torch.empty_like(s["q"])
        s["max_q"], s["max_kv"] = max(s["new"]), max(s["kv_lens"])
        n = L.qe_attention_workspace_bytes(s["cache_handle"], s["heads"], s["T"], s["seqs"], s["max_q"], s["max_kv"])
        s["ws"] = empty(max(n, 256), dtype=torch.uint8)
    if op == "verify":
        s["taken"], s["next"] = empty(s["seqs"], dtype=torch.int32), empty(s["seqs"], dtype=torch.int32)
        s["path"] = empty(s["N"], dtype=torch.int32)
        s["ws"] = empty(max(L.qe_verify_workspace_bytes(s["seqs"], s["vocab"]), 256), dtype=torch.uint8)


def _run_own(s):
    from quantized_linear_moe_amd import libqe as L
    op = s["op"]
    if op == "rope":
        L.qe_rope_apply(s["rope"], s["pos"], s["input"], s["out"])
        return {"y": s["out"]}
    if op == "append":
        L.qe_kv_append(s["cache_handle"], s["k_in"], s["v_in"], s["slot"], rope=s["rope"], pos=s["pos"], q=s["q_in"],
                       q_out=s["q_out"])
        out = {"q": s["q_out"]} if s["heads"] else {}
        for i, name in enumerate(("k", "v")):
            out[name] = s[name]
            if s["cache"] == "i8":
                out[name] = torch.mul(s[name], s[name + "_scale"][..., None], out=s["values"][i])
        return out
    if op == "attn":
        L.qe_attention(s["cache_handle"], s["q"], s["q_start"], s["kv_len"], s["pages"], s["max_q"], s["max_kv"],
                       s["out"], s["ws"], tree=s["tree_bits"])
        return {"o": s["out"]}
    L.qe_verify_drafts(s["p"], s["row_start"], s["token"], s["u"], s["taken"], s["path"], s["next"], s["ws"],
                       draft_p=s["draft_p"], parent=s["parent"], max_rows=max(s["rows_of"]))
    return {"taken": s["taken"], "path": s["path"], "next": s["next"]}


# -------------------------------------------------------------------- plain forms
def _angles(s):
    """float64 angles [T][rot/2]: every pair's position row times its frequency."""
    pos = s["pos"].double()
    if not s["sections"]:
        return pos[0][:, None] * s["inv_freq"]
    row = torch.repeat_interleave(torch.arange(3, device=DEV), torch.tensor(_sections(s), device=DEV))
    return pos[row].t() * s["inv_freq"]


def _rotate(s, x, dtype):
    """x [T][heads][hd] with its first rot channels rotated, in `dtype`."""
    a, rot = _angles(s), s["rot"]
    c = (torch.cos(a) * s["scale"]).to(dtype)[:, None]
    n = (torch.sin(a) * s["scale"]).to(dtype)[:, None]
    x = x.to(dtype)
    y = x.clone()
    if s["layout"] == "half":
        first, second = slice(0, rot // 2), slice(rot // 2, rot)
    else:
        first, second = slice(0, rot, 2), slice(1, rot, 2)
    x1, x2 = x[..., first], x[..., second]
    y[..., first] = x1 * c - x2 * n
    y[..., second] = x2 * c + x1 * n
    return y


def _codes8(x):
    """The values that 8-bit codes of every row's last axis stand for, in x's type."""
    scale = x.abs().amax(-1, keepdim=True) / 127
    return torch.round(x / torch.where(scale > 0, scale, 1.0)).clamp_(-127, 127) * scale


def _append(s, dtype):
    """Both caches' values after the call, and q, in `dtype` (codes are made from 32-bit values)."""
    k, v = _rotate(s, s["k_in"], dtype), s["v_in"].to(dtype)
    q = _rotate(s, s["q_in"], dtype) if s["heads"] else None
    at = torch.nonzero(s["slot"] >= 0)[:, 0]
    slot = s["slot"][at].long()
    out = {"q": q} if s["heads"] else {}
    for name, x in (("k", k), ("v", v)):
        cache = s[name].to(dtype)
        if s["cache"] == "i8":
            cache = cache * s[name + "_scale"][..., None].to(dtype)
            x = _codes8(x.float().to(dtype))
        cache[slot // s["page"], :, slot % s["page"]] = x[at]
        out[name] = cache
    return out


def _attention(s, dtype):
    """softmax(q K^T / sqrt(hd)) V per sequence and key head over the keys each token sees, in `dtype`."""
    group, hd, page = s["heads"] // s["kv_heads"], s["hd"], s["page"]
    out = torch.empty(s["q"].shape, dtype=dtype, device=DEV)
    t = 0
    for b, (n, L) in enumerate(zip(s["new"], s["kv_lens"])):
        pages = s["pages"][b, : (L + page - 1) // page].long()
        rel = torch.arange(L, device=DEV) - (L - n)  # number of the new token that a key belongs to
        if s["tree_bits"] is None:
            seen = rel[None] <= torch.arange(n, device=DEV)[:, None]
        else:
            word = s["tree_bits"][t : t + n][:, rel.clamp(min=0) // 32]
            seen = (rel[None] < 0) | (((word >> (rel.clamp(min=0) % 32)) & 1) == 1)
        for h in range(s["kv_heads"]):
            kv = []
            for name in ("k", "v"):
                x = s[name][pages, h].to(dtype)
                if s["cache"] == "i8":
                    x = x * s[name + "_scale"][pages, h][..., None].to(dtype)
                kv.append(x.reshape(-1, hd)[:L])
            q = s["q"][t : t + n, h * group : (h + 1) * group].to(dtype).transpose(0, 1)
            z = torch.matmul(q, kv[0].t().contiguous()) / math.sqrt(hd)
            z = z.masked_fill_(~seen, -math.inf)
            e = torch.exp(z - z.amax(-1, keepdim=True))
            o = torch.matmul(e / e.sum(-1, keepdim=True), kv[1])
            out[t : t + n, h * group : (h + 1) * group] = o.transpose(0, 1)
        t += n
    return out


def _verify(s):
    """The walk over the drafts and the draw after it; the draw's sums in 64 bits."""
    row = torch.arange(s["N"], device=DEV)
    starts = [0]
    for n in s["rows_of"]:
        starts.append(starts[-1] + n)
    first = torch.repeat_interleave(torch.tensor(starts[:-1], device=DEV), torch.tensor(s["rows_of"], device=DEV))
    above = first + torch.tensor(s["parents"], device=DEV).clamp(min=0)
    token = s["token"].long()
    p_token = s["p"][above, token].double().tolist()  # the target's probability of every draft, where it hangs
    q_token = s["draft_p"][row, token].double().tolist() if s["draft_p"] is not None else None
    u, tok = s["u"].double().tolist(), s["token"].tolist()
    taken, path, rows_p, rows_q, dropped = [], [], [], [], []
    for b, n in enumerate(s["rows_of"]):
        at, cur, steps, reject = starts[b], 0, [], []
        while True:
            rest, reject, hit = 1.0, [], None
            for i in range(cur + 1, n):
                if s["parents"][at + i] != cur:
                    continue
                if q_token is not None:
                    ok = u[at + i] * q_token[at + i] < p_token[at + i]
                else:
                    ok = tok[at + i] not in [tok[at + r] for r in reject] and u[at + i] * rest < p_token[at + i]
                if ok:
                    hit = i
                    break
                if q_token is None and tok[at + i] not in [tok[at + r] for r in reject]:
                    rest -= p_token[at + i]
                reject.append(i)
            if hit is None:
                break
            steps.append(hit)
            cur = hit
        taken.append(len(steps))
        path += steps + [-1] * (n - len(steps))
        rows_p.append(at + cur)
        rows_q.append(at + reject[0] if q_token is not None and reject else -1)
        dropped += [(b, tok[at + r]) for r in reject]
    R = s["p"][torch.tensor(rows_p, device=DEV)].double()
    if q_token is not None:
        at = torch.tensor(rows_q, device=DEV)
        R = torch.where((at >= 0)[:, None], (R - s["draft_p"][at.clamp(min=0)].double()).clamp_(min=0), R)
    elif dropped:
        d = torch.tensor(dropped, device=DEV)
        R[d[:, 0], d[:, 1]] = 0.0
    C = torch.cumsum(R, -1)
    goal = s["u"][torch.tensor(starts[:-1], device=DEV)].double()[:, None] * C[:, -1:]
    nxt = torch.searchsorted(C, goal, right=True)[:, 0].clamp(max=s["vocab"] - 1)
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device=DEV)  # noqa: E731
    return {"taken": i32(taken), "path": i32(path), "next": nxt.to(torch.int32)}


def _run_plain(s):
    op = s["op"]
    if op == "rope":
        return {"y": _rotate(s, s["input"], torch.float32).to(s["input"].dtype)}
    if op == "append":
        return {k: v.to(torch.bfloat16) for k, v in _append(s, torch.float32).items()}
    if op == "attn":
        return {"o": _attention(s, torch.float32).to(torch.bfloat16)}
    return _verify(s)


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ------------------------------------------------------------------- work, exact
def work(case):
    op = case["op"]
    if op == "verify":
        b = case["seqs"] * case["vocab"] * 4 * (1 if case["tree"] else 2)
        return {"bytes": b, "flops": 3.0 * case["seqs"] * case["vocab"]}
    hd = case["hd"]
    if op == "attn":
        new, kv = _lengths(case)
        T, keys = sum(new), sum(kv)
        # a token of a tree sees its ancestors, a handful; a token of a text all before it
        pairs = sum(n * (k - n) + (n * (n + 1) / 2 if not case["tree"] else n * min(n, 6)) for n, k in zip(new, kv))
        per_key = 2 * case["kv_heads"] * (hd * 2 if case["cache"] == "bf16" else hd + 4)
        return {"bytes": keys * per_key + T * case["heads"] * hd * 4, "flops": 4.0 * pairs * case["heads"] * hd}
    e = 2 if case["x"] == "bf16" else 4
    if op == "rope":
        n = case["T"] * case["heads"] * hd
        return {"bytes": 2 * n * e, "flops": 3.0 * n}
    n_q, n_kv = case["T"] * case["heads"] * hd, 2 * case["T"] * case["kv"] * hd
    b = n_q * (e + 2) + n_kv * (e + (2 if case["cache"] == "bf16" else 1 + 4 / hd))
    return {"bytes": b, "flops": 3.0 * (n_q + n_kv)}


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    f64 = torch.float64
    if op == "verify":
        return None
    if op == "append":
        out = {}
        turn = _turns(s)
        k, v = _turned(s, s["k_in"], turn), s["v_in"].to(f64)
        if s["heads"]:
            out["q"] = _turned(s, s["q_in"], turn)
        for name, x in (("k", k), ("v", v)):
            if s["cache"] == "i8":  # the values that get codes are held in 32 bits
                x = x.float().to(f64)
                step = x.abs().amax(-1, keepdim=True) / 127
                x = torch.where(step > 0, torch.round(x / step.clamp(min=1e-300)) * step, 0.0)
                out[name] = s[name].to(f64) * s[name + "_scale"].to(f64)[..., None]
            else:
                out[name] = s[name].to(f64)
            for t, slot in enumerate(s["slot"].tolist()):
                if slot >= 0:
                    out[name][slot // s["page"], :, slot % s["page"]] = x[t]
        return out
    if op == "rope":
        return {"y": _turned(s, s["input"], _turns(s))}
    return {"o": _exact_attention(s)}


def _turns(s):
    """exp(i angle) of every token and pair."""
    T, pairs = s["pos"].shape[1], s["rot"] // 2
    turn = torch.empty(T, pairs, dtype=torch.float64, device=DEV)
    lo = 0
    for row, width in enumerate(_sections(s) or (pairs,)):
        turn[:, lo : lo + width] = torch.outer(s["pos"][row].double(), s["inv_freq"][lo : lo + width])
        lo += width
    return torch.polar(torch.full_like(turn, float(s["scale"])), turn)


def _turned(s, x, turn):
    """The first rot channels of x as complex numbers, times exp(i angle)."""
    x = x.double()
    part = x[..., : s["rot"]]
    if s["layout"] == "half":
        z = torch.complex(*part.chunk(2, -1)) * turn[:, None]
        part = torch.cat((z.real, z.imag), -1)
    else:
        z = torch.view_as_complex(part.reshape(*part.shape[:-1], -1, 2).contiguous()) * turn[:, None]
        part = torch.view_as_real(z).flatten(-2)
    return torch.cat((part, x[..., s["rot"] :]), -1)


def _exact_attention(s):
    """Every new token's softmax over the keys it sees, all heads of a piece of tokens at once."""
    group, page, hd = s["heads"] // s["kv_heads"], s["page"], s["hd"]
    out = torch.empty(s["q"].shape, dtype=torch.float64, device=DEV)
    base = 0
    for b in range(s["seqs"]):
        n, L = s["new"][b], s["kv_lens"][b]
        key = torch.arange(L, device=DEV)
        where = s["pages"][b].long()[key // page]
        K, V = (s[c][where, :, key % page].double() for c in ("k", "v"))  # [L][kv heads][hd]
        if s["cache"] == "i8":
            K = K * s["k_scale"][where, :, key % page].double()[..., None]
            V = V * s["v_scale"][where, :, key % page].double()[..., None]
        K, V = K.permute(1, 2, 0).contiguous(), V.permute(1, 0, 2).contiguous()
        for lo in range(0, n, 256):
            hi = min(n, lo + 256)
            q = s["q"][base + lo : base + hi].double().reshape(hi - lo, s["kv_heads"], group * hd)
            q = q.reshape(hi - lo, s["kv_heads"], group, hd).permute(1, 0, 2, 3).reshape(s["kv_heads"], -1, hd)
            z = torch.bmm(q.contiguous(), K) * hd ** -0.5
            for i in range(lo, hi):
                if s["tree_bits"] is None:
                    hidden = key > L - n + i
                else:
                    words = s["tree_bits"][base + i]
                    new = torch.stack([(words >> bit) & 1 for bit in range(32)], 1).flatten()[:n] == 1
                    hidden = torch.cat((torch.zeros(L - n, dtype=torch.bool, device=DEV), ~new))
                z[:, (i - lo) * group : (i - lo + 1) * group, hidden] = -math.inf
            o = torch.bmm(torch.softmax(z, -1), V)
            out[base + lo : base + hi] = o.reshape(s["kv_heads"], hi - lo, group, hd).permute(1, 0, 2, 3).reshape(
                hi - lo, s["heads"], hd)
        base += n
    return out
