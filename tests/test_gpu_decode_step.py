"""The operators of a decoding step together, as a program runs them: quantized q, k and v linears, the append with the
rotation on the way, the attention over the cache, the output linear, and the verification of drafts; prompts, single
tokens and trees over one growing cache, on streams and in captured graphs.

The attention of a whole prompt and of the same tokens in pieces or one by one is the same sum in another order, each
within the attention's own bound of the definition: they differ by at most twice that.
"""

import numpy as np
import pytest
import torch

from oracle import qe_cache_oracle as C
from oracle import qe_oracle as O

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF = torch.bfloat16


@pytest.fixture(scope="module")
def Q():
    import quantized_linear_moe_amd as q
    return q


class Layer:
    """q, k, v and o linears of one layer with their cache."""

    def __init__(self, Q, heads=8, kv=2, hd=64, hidden=256, page=16, pages=24, i8=False, seed=0):
        self.L, self.heads, self.kv, self.hd, self.hidden, self.page = Q.libqe, heads, kv, hd, hidden, page
        rng = np.random.default_rng(seed)
        self.lins = {}
        for name, d_in, d_out in (("q", hidden, heads * hd), ("k", hidden, kv * hd), ("v", hidden, kv * hd),
                                  ("o", heads * hd, hidden)):
            params = {"W_f": (rng.standard_normal((d_out, d_in)) / d_in ** 0.5).astype(np.float32), "s": None}
            self.lins[name] = Q.QELinear.from_params(params, 4, 8, device=DEV)
        shape = (pages, kv, page, hd)
        if i8:
            self.store = [torch.zeros(shape, dtype=torch.int8, device=DEV) for _ in range(2)]
            self.store += [torch.full(shape[:3], float("nan"), device=DEV) for _ in range(2)]
        else:
            self.store = [torch.full(shape, float("nan"), dtype=BF, device=DEV) for _ in range(2)]
        self.cache = self.L.make_cache(*self.store)
        f, _ = self.L.qe_rope_freqs(hd, 1e4)
        self.rope = self.L.make_rope(torch.from_numpy(f).to(DEV))

    def step(self, x, pos, slot, q_start, kv_len, pages, max_q, max_kv, tree=None, rows=None, stream=None):
        """x [T, hidden] bf16 through the layer; returns (attention rows, y)."""
        L, T = self.L, x.shape[0]
        q, k, v = (self.lins[n].forward(x).unflatten(1, (-1, self.hd)) for n in ("q", "k", "v"))
        qr = torch.empty(T, self.heads, self.hd, dtype=BF, device=DEV)
        L.qe_kv_append(self.cache, k, v, slot, rope=self.rope, pos=pos, q=q, q_out=qr)
        o = torch.zeros(T, self.heads, self.hd, dtype=BF, device=DEV) if rows is None else rows
        n = L.qe_attention_workspace_bytes(self.cache, self.heads, T, kv_len.shape[0], max_q, max_kv)
        ws = torch.empty(max(n, 16), dtype=torch.uint8, device=DEV)
        L.qe_attention(self.cache, qr, q_start, kv_len, pages, max_q, max_kv, o, ws, tree=tree)
        self.last = (q, k, v, qr)
        return o, self.lins["o"].forward(o.flatten(1))


def _i32(a):
    return torch.tensor(a, dtype=torch.int32, device=DEV)


def _tokens(layer, T, seed=1):
    return torch.randn(T, layer.hidden, generator=torch.Generator().manual_seed(seed)).to(BF).to(DEV)


def _bound(o, A, n):
    return 2.0 ** -8 * np.abs(o) + 1.01 * A * (2 * 2.0 ** -8 + 2.0 ** -9 + 2 * n * 2.0 ** -23)


@pytest.mark.parametrize("i8", [False, True])
def test_prompt_then_tokens(Q, i8):
    """A prompt at once, its end again token by token and as a chain tree: the same rows; and against the definition on
    what the cache holds."""
    T, cut = 70, 64
    a, b = Layer(Q, i8=i8), Layer(Q, i8=i8)
    table = torch.randperm(24, generator=torch.Generator().manual_seed(2))[:5].to(torch.int32).to(DEV)
    x, pos = _tokens(a, T), _i32(range(T))
    t = torch.arange(T, device=DEV)
    slot = (table.long()[t // 16] * 16 + t % 16).to(torch.int32)
    whole, _ = a.step(x, pos, slot, _i32([0, T]), _i32([T]), table[None], T, T)
    q, k, v, qr = a.last

    # the definition, on the cache's own values
    place = slot.long()
    K, V = (s[place // 16, :, place % 16].float() for s in a.store[:2])
    if i8:
        K, V = (c * s[place // 16, :, place % 16][..., None] for c, s in zip((K, V), a.store[2:]))
        codes, scales = O.quant_act(v.cpu().numpy().reshape(-1, 64), None, 8)  # what the linear wrote, in 8 bits
        assert np.array_equal(a.store[1][place // 16, :, place % 16].cpu().numpy().reshape(-1, 64), codes)
    else:
        assert torch.equal(V, v.to(BF).float())
    o, A, _ = C.attention(qr.float().cpu().numpy(), K.cpu().numpy(), V.cpu().numpy(), C.sees(T, 0, T), 64 ** -0.5)
    assert np.all(np.abs(whole.float().cpu().numpy() - o) <= _bound(o, A, T))

    b.step(x[:cut], pos[:cut], slot[:cut], _i32([0, cut]), _i32([cut]), table[None], cut, cut)
    for i in range(cut, T):
        row, _ = b.step(x[i:i + 1], pos[i:i + 1], slot[i:i + 1], _i32([0, 1]), _i32([i + 1]), table[None], 1, 4096)
        assert np.all(np.abs(row.float().cpu().numpy() - whole[i:i + 1].float().cpu().numpy()) <=
                      2 * _bound(o[i:i + 1], A[i:i + 1], T))
    bits = _i32([(2 << i) - 1 for i in range(T - cut)])[:, None].contiguous()
    rows, _ = b.step(x[cut:], pos[cut:], slot[cut:], _i32([0, T - cut]), _i32([T]), table[None], T - cut, T, tree=bits)
    assert np.all(np.abs(rows.float().cpu().numpy() - whole[cut:].float().cpu().numpy()) <= 2 * _bound(o[cut:], A[cut:], T))


def test_draft_tree_step_is_its_branches(Q):
    """A token of a draft tree gets the row that its branch alone would have got; the walk then keeps one branch, whose
    entries move to the places behind the text, and the next step goes on from there."""
    a = Layer(Q)
    L = a.L
    ctx, par = 37, [-1, 0, 0, 1, 2, 2, 4]  # row 0: the last accepted token
    n = len(par)
    depth = [0] * n
    for i in range(1, n):
        depth[i] = depth[par[i]] + 1
    table = _i32([[3, 7, 1, 12, 0]])
    x = _tokens(a, ctx + n, 3)
    t = torch.arange(ctx + n, device=DEV)
    slot = (table[0].long()[t // 16] * 16 + t % 16).to(torch.int32)
    pos = _i32(list(range(ctx)) + [ctx + d for d in depth])
    a.step(x[:ctx], pos[:ctx], slot[:ctx], _i32([0, ctx]), _i32([ctx]), table, ctx, ctx)
    bits = [1]
    for i in range(1, n):
        bits.append(bits[par[i]] | 1 << i)
    rows, _ = a.step(x[ctx:], pos[ctx:], slot[ctx:], _i32([0, n]), _i32([ctx + n]), table, n, ctx + n,
                     tree=_i32(bits)[:, None].contiguous())
    for leaf in (3, 5, 6):
        path = [leaf]
        while par[path[0]] >= 0:
            path.insert(0, par[path[0]])
        b = Layer(Q)
        take = list(range(ctx)) + [ctx + i for i in path]
        m = len(take)
        alone, _ = b.step(x[take], pos[take], slot[:m], _i32([0, m]), _i32([m]), table, m, m)
        # (the same keys in other places, so another order of float32 sums; weights rounded to bf16 as before)
        K, V = (s[slot[:m].long() // 16, :, slot[:m].long() % 16].float().cpu().numpy() for s in b.store)
        o, A, _ = C.attention(b.last[3].float().cpu().numpy(), K, V, C.sees(m, 0, m), 64 ** -0.5)
        got = rows[path].float().cpu().numpy()
        assert np.all(np.abs(got - alone[ctx:].float().cpu().numpy()) <= 2 * _bound(o[ctx:], A[ctx:], m))

    rng = np.random.default_rng(0)
    V = 500
    e = np.exp(2 * rng.standard_normal((n, V)))
    p = (e / e.sum(1, keepdims=True)).astype(np.float32)
    tok = np.array([0] + [int(np.argsort(-p[par[i]])[par[:i].count(par[i])]) for i in range(1, n)], np.int32)
    u = np.array([0.4, 0.99, 0.0, 0.0, 0.0, 0.5, 0.0], np.float32)
    taken, nxt, path = _i32([0]), _i32([0]), _i32([0] * n)
    ws = torch.empty(L.qe_verify_workspace_bytes(1, V), dtype=torch.uint8, device=DEV)
    L.qe_verify_drafts(torch.from_numpy(p).to(DEV), _i32([0, n]), _i32(tok), torch.from_numpy(u).to(DEV), taken, path, nxt,
                       ws, parent=_i32(par), max_rows=n)
    want, token = C.verify(p, tok, u, parent=par)
    assert want and int(taken) == len(want) and path.tolist()[:len(want)] == want and int(nxt) == token

    # the accepted branch moves to the places behind the text
    keep = [0] + want
    src, dst = slot[ctx:].long()[keep], slot[ctx:].long()[:len(keep)]
    for s in a.store:
        s[dst // 16, :, dst % 16] = s[src // 16, :, src % 16].clone()
    m = ctx + len(keep)
    x_next = _tokens(a, 1, 9)
    row, _ = a.step(x_next, _i32([m]), slot[m:m + 1], _i32([0, 1]), _i32([m + 1]), table, 1, 128)
    b = Layer(Q)
    take = list(range(ctx)) + [ctx + i for i in keep]
    b.step(x[take], _i32(range(m)), slot[:m], _i32([0, m]), _i32([m]), table, m, m)
    alone, _ = b.step(x_next, _i32([m]), slot[m:m + 1], _i32([0, 1]), _i32([m + 1]), table, 1, 128)
    assert torch.equal(row, alone)


def test_padded_batch(Q):
    """A batch padded to a fixed count of tokens and sequences: padding has no place, and its rows are left."""
    a = Layer(Q)
    T, pad = 5, 3
    x = _tokens(a, T + pad, 4)
    slot = _i32([0, 1, 16, 17, 18] + [-1] * pad)
    pages = _i32([[0], [1], [999999]])
    rows = torch.full((T + pad, 8, 64), 77.0, dtype=BF, device=DEV)
    a.step(x, _i32([0, 1, 0, 1, 2] + [0] * pad), slot, _i32([0, 2, T, T]), _i32([2, 3, 0]), pages, 4, 16, rows=rows)
    assert bool((rows[T:] == 77).all())
    b = Layer(Q)
    alone, _ = b.step(x[2:T], _i32([0, 1, 2]), slot[2:T], _i32([0, 3]), _i32([3]), pages[1:2], 4, 16)
    assert torch.equal(rows[2:T], alone)
    assert bool(torch.isnan(a.store[0][2:]).all())  # nothing of the padding was stored


def _operators(Q, seed, long=2000):
    """One call of each operator over buffers of their own, its inputs (to change in place) and outputs."""
    L = Q.libqe
    g = torch.Generator().manual_seed(seed)
    f, _ = L.qe_rope_freqs(64, 1e4)
    rope = L.make_rope(torch.from_numpy(f).to(DEV))
    T, heads, kv, hd, pages, page = 3, 8, 2, 64, 140, 16
    k, v = (torch.randn(pages, kv, page, hd, generator=g).to(BF).to(DEV) for _ in range(2))
    cache = L.make_cache(k, v)
    x = [torch.randn(T, h, hd, generator=g).to(BF).to(DEV) for h in (heads, kv, kv)]
    table = torch.randperm(pages, generator=g).to(torch.int32).to(DEV)[None, :130].contiguous()
    kv_len, q_start = _i32([long]), _i32([0, T])
    j = torch.arange(long - T, long, device=DEV)
    slot = (table[0].long()[j // page] * page + j % page).to(torch.int32)
    pos = j.to(torch.int32)
    qr, out = torch.empty_like(x[0]), torch.empty_like(x[0])
    ws = torch.empty(max(L.qe_attention_workspace_bytes(cache, heads, T, 1, T, 2080), 16), dtype=torch.uint8, device=DEV)
    y = torch.empty_like(x[0])
    p = torch.softmax(3 * torch.randn(6, 9000, generator=g), -1).to(DEV)
    d = torch.softmax(3 * torch.randn(6, 9000, generator=g), -1).to(DEV)
    tok = torch.randint(0, 9000, (6,), generator=g, dtype=torch.int32).to(DEV)
    u = torch.rand(6, generator=g).to(DEV)
    taken, nxt, path = _i32([0, 0]), _i32([0, 0]), _i32([0] * 6)
    vws = torch.empty(L.qe_verify_workspace_bytes(2, 9000), dtype=torch.uint8, device=DEV)

    def call():
        L.qe_rope_apply(rope, pos, x[0], y)
        L.qe_kv_append(cache, x[1], x[2], slot, rope=rope, pos=pos, q=x[0], q_out=qr)
        L.qe_attention(cache, qr, q_start, kv_len, table, T, 2080, out, ws)
        L.qe_verify_drafts(p, _i32_keep, tok, u, taken, path, nxt, vws, draft_p=d, max_rows=6)
    _i32_keep = _i32([0, 4, 6])
    return call, x + [p, d, u], [y, qr, k, v, out, taken, path, nxt]


def test_captured_and_replayed(Q):
    """The four operators captured once and replayed over changed inputs, with eager calls in between."""
    call, inputs, outputs = _operators(Q, 1)
    other, _, _ = _operators(Q, 2)
    call()
    torch.cuda.synchronize()
    first = [t.clone() for t in outputs]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for turn in range(4):
        if turn:
            g = torch.Generator().manual_seed(turn)
            for t in inputs[:3]:
                t.copy_(torch.randn(t.shape, generator=g).to(t.dtype))
            inputs[3].copy_(torch.softmax(3 * torch.randn(inputs[3].shape, generator=g), -1))
            inputs[5].copy_(torch.rand(inputs[5].shape, generator=g))
        for t in (outputs[0], outputs[1], outputs[4]):
            t.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        replayed = [t.clone() for t in outputs]
        if not turn:
            assert all(torch.equal(a, b) for a, b in zip(replayed, first))
        other()  # eager work between the replays
        call()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(replayed, outputs)), turn


def test_captured_call_serves_growing_lengths(Q):
    """One captured attention, replayed while the sequence grows from nothing through single pieces to many."""
    L = Q.libqe
    heads, kv, hd, page = 8, 2, 128, 16
    g = torch.Generator().manual_seed(3)
    k, v = (torch.randn(300, kv, page, hd, generator=g).to(BF).to(DEV) for _ in range(2))
    cache = L.make_cache(k, v)
    q = torch.randn(1, heads, hd, generator=g).to(BF).to(DEV)
    table = torch.arange(300, dtype=torch.int32, device=DEV)[None]
    kv_len, q_start, out = _i32([1]), _i32([0, 1]), torch.empty_like(q)
    ws = torch.empty(L.qe_attention_workspace_bytes(cache, heads, 1, 1, 1, 4800), dtype=torch.uint8, device=DEV)
    L.qe_attention(cache, q, q_start, kv_len, table, 1, 4800, out, ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        L.qe_attention(cache, q, q_start, kv_len, table, 1, 4800, out, ws)
    for n in (0, 1, 5, 128, 129, 600, 3000, 4800, 17):
        kv_len.fill_(n)
        out.fill_(77.0)
        ws.fill_(255)
        graph.replay()
        torch.cuda.synchronize()
        K, V = (t.transpose(1, 2).reshape(-1, kv, hd)[:n].float().cpu().numpy() for t in (k, v))
        o, A, _ = C.attention(q.float().cpu().numpy(), K, V, np.ones((1, n), bool), hd ** -0.5)
        assert np.all(np.abs(out.float().cpu().numpy() - o) <= _bound(o, A, max(n, 1))), n


def test_two_streams(Q):
    """Two programs on streams of their own, with workspaces of their own, at the same time."""
    calls = [_operators(Q, s) for s in (1, 2)]
    want = []
    for call, _, outputs in calls:
        call()
        torch.cuda.synchronize()
        want.append([t.clone() for t in outputs])
    streams = [torch.cuda.Stream() for _ in calls]
    for _ in range(10):
        for (call, _, _), s in zip(calls, streams):
            with torch.cuda.stream(s):
                call()
    torch.cuda.synchronize()
    for (_, _, outputs), w in zip(calls, want):
        assert all(torch.equal(a, b) for a, b in zip(outputs, w))


def test_bindings_refuse_mixed_devices(Q):
    L = Q.libqe
    k = torch.zeros(4, 2, 16, 64, dtype=BF, device=DEV)
    cache = L.make_cache(k, k.clone())
    x = torch.zeros(2, 2, 64, dtype=BF, device=DEV)
    with pytest.raises(ValueError, match="not on device"):
        L.qe_kv_append(cache, x, x.cpu(), _i32([0, 1]))
    with pytest.raises(ValueError, match="not on device"):
        L.qe_attention(cache, x, _i32([0, 2]).cpu(), _i32([2]), _i32([[0]]), 2, 16, x.clone(), None)
    with pytest.raises(ValueError, match="not on device"):
        L.make_cache(k, k.cpu())
    rope = L.make_rope(torch.zeros(32, dtype=torch.float64))
    with pytest.raises(ValueError, match="inv_freq is on"):
        L.qe_rope_apply(rope, _i32([0, 1]), x, x)
    with pytest.raises(ValueError, match="inv_freq is on"):
        L.qe_kv_append(cache, x, x, _i32([0, 1]), rope=rope, pos=_i32([0, 1]))
