"""GPU parity of the verification of drafts.  Probabilities are float32 and both sides compare and sum in float64; the
order of a sum moves it by less than 2^-40 of itself at these sizes, and no random number here lies that close to a border,
so accepted rows and drawn tokens are equal."""

import numpy as np
import pytest
import torch

from oracle import qe_cache_oracle as C

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module")
def L():
    from quantized_linear_moe_amd import libqe
    return libqe


def _soft(rng, n, V, spread):
    z = spread * rng.standard_normal((n, V))
    e = np.exp(z - z.max(1, keepdims=True))
    return (e / e.sum(1, keepdims=True)).astype(np.float32)


def _case(rng, rows, V, kind, spread=3.0):
    """rows: per sequence; kind: drawn (chain with distributions), chain, tree (chosen tokens)."""
    N = sum(rows)
    p = _soft(rng, N, V, spread)
    d = parent = None
    tok = np.zeros(N, np.int32)
    first = np.repeat(np.cumsum([0] + rows)[:-1], rows)
    local = np.arange(N) - first
    above = np.maximum(local - 1, 0)
    if kind == "tree":
        above = np.array([rng.integers(max(0, i - 5), i) if i else 0 for i in local])
        parent = np.where(local > 0, above, -1).astype(np.int32)
    if kind == "drawn":
        d = np.sqrt(np.roll(p, 1, 0) * _soft(rng, N, V, spread))
        d = (d / d.sum(1, keepdims=True)).astype(np.float32)
    for i in range(N):
        w = p[first[i] + above[i]] if d is None else d[i]
        best = np.argsort(-w)[:4]
        tok[i] = rng.choice(best) if d is None else rng.choice(V, p=w.astype(np.float64) / w.astype(np.float64).sum())
    u = rng.random(N).astype(np.float32)
    return p, d, tok, u, parent


def _run(L, rows, p, d, tok, u, parent, tail=0, pad=0, max_rows=None):
    N, V = p.shape
    n = len(rows)
    i32 = lambda a: torch.tensor(np.asarray(a), dtype=torch.int32, device=DEV)  # noqa: E731

    def dist(a):
        if a is None:
            return None
        wide = torch.full((N, V + pad), float("nan"), device=DEV)
        wide[:, :V] = torch.from_numpy(a)
        return wide[:, :V]
    taken, nxt, path = (torch.full((k,), 77, dtype=torch.int32, device=DEV) for k in (n, n, N))
    ws = torch.full((L.qe_verify_workspace_bytes(n, V),), 255, dtype=torch.uint8, device=DEV)
    L.qe_verify_drafts(dist(p), i32(np.cumsum([0] + rows)), i32(tok), torch.from_numpy(u).to(DEV), taken, path, nxt, ws,
                       draft_p=dist(d), parent=None if parent is None else i32(parent),
                       max_rows=max(rows) if max_rows is None else max_rows)
    torch.cuda.synchronize()
    return taken.cpu().numpy(), path.cpu().numpy(), nxt.cpu().numpy()


def _check(rows, p, d, tok, u, parent, got):
    taken, path, nxt = got
    at, seen = 0, []
    for s, n in enumerate(rows):
        cut = slice(at, at + n)
        if n == 0:
            assert taken[s] == 0 and nxt[s] == -1
            continue
        want, token = C.verify(p[cut], tok[cut], u[cut], None if d is None else d[cut],
                               None if parent is None else parent[cut])
        assert taken[s] == len(want), s
        assert list(path[cut]) == want + [-1] * (n - len(want)), s
        assert nxt[s] == token, s
        seen.append(len(want))
        at += n
    return seen


@pytest.mark.parametrize("kind", ["drawn", "chain", "tree"])
@pytest.mark.parametrize("V", [1, 2, 7, 255, 1000, 4096, 4097, 32003])
@pytest.mark.parametrize("rows", [[1], [5], [1, 2, 9], [33, 1, 64, 65]])
def test_verify(L, rows, V, kind):
    rng = np.random.default_rng(V + len(rows) + len(kind))
    for spread in (0.5, 4.0):
        a = _case(rng, rows, V, kind, spread)
        _check(rows, *a, _run(L, rows, *a, pad=3 * (V % 2)))


@pytest.mark.parametrize("kind", ["drawn", "chain", "tree"])
def test_many_small_walks(L, kind):
    """Thousands of walks over a few tokens, of every length; the accepted counts vary."""
    rng = np.random.default_rng(11)
    rows = [int(n) for n in rng.integers(0, 7, 3000)]
    a = _case(rng, rows, 5, kind, 1.0)
    seen = _check(rows, *a, _run(L, rows, *a))
    assert len(set(seen)) >= 4


def test_large_trees(L):
    rng = np.random.default_rng(5)
    rows = [1024, 700]
    a = _case(rng, rows, 50, "tree", 1.0)
    _check(rows, *a, _run(L, rows, *a))


def test_all_accepted_and_none(L):
    for kind in ("drawn", "chain", "tree"):
        for level in (0.0, float(np.float32(1 - 2.0 ** -24))):
            rng = np.random.default_rng(3)
            p, d, tok, u, parent = _case(rng, [40, 3], 300, kind)
            u[:] = level
            _check([40, 3], p, d, tok, u, parent, _run(L, [40, 3], p, d, tok, u, parent))


def test_repeated_siblings_and_bad_rows(L):
    """The same token twice under one parent, tokens outside the vocabulary, parents that are not below their row."""
    rng = np.random.default_rng(8)
    for _ in range(20):
        rows = [12]
        p, d, tok, u, parent = _case(rng, rows, 6, "tree", 1.0)
        parent[1:7] = 0
        tok[1:7] = rng.integers(0, 3, 6)
        tok[3], tok[8], parent[9], parent[10] = -1, 6, 9, -4
        want = parent.copy()
        want[9] = -1  # (not a child of any row)
        got = _run(L, rows, p, d, tok, u, parent)
        _check(rows, p, d, tok, u, want, got)
        p, d, tok, u, _ = _case(rng, rows, 6, "drawn", 1.0)
        tok[4] = 2 ** 31 - 1
        _check(rows, p, d, tok, u, None, _run(L, rows, p, d, tok, u, None))


def test_nothing_left_to_draw_from(L):
    """One-hot rows whose token is refused draw from the row itself; rows of zeros and of NaN give -1."""
    p = np.zeros((3, 10), np.float32)
    p[:, 4] = 0.5  # not normalised: 0.5 is refused by u = 0.9
    tok = np.array([0, 4, 4], np.int32)
    u = np.array([0.3, 0.9, 0.9], np.float32)
    taken, path, nxt = _run(L, [3], p, None, tok, u, None)
    assert taken[0] == 0 and nxt[0] == 4
    for v in (0.0, np.nan):
        taken, path, nxt = _run(L, [3], np.full((3, 10), v, np.float32), None, tok, u, None)
        assert taken[0] == 0 and nxt[0] == -1 and list(path) == [-1] * 3
        taken, path, nxt = _run(L, [3], np.full((3, 10), v, np.float32), np.full((3, 10), 0.1, np.float32), tok, u, None)
        assert taken[0] == 0 and nxt[0] == -1


def test_more_rows_than_said(L):
    """Rows past max_rows are left out; starts past the rows are cut."""
    rng = np.random.default_rng(2)
    p, d, tok, u, parent = _case(rng, [9], 40, "chain")
    u[1:] = 0.0
    taken, path, nxt = _run(L, [9], p, d, tok, u, parent, max_rows=4)
    assert taken[0] == 3 and list(path[:4]) == [1, 2, 3, -1] and np.all(path[4:] == 77)
    want = C.verify(p[:4], tok[:4], u[:4])
    assert (list(path[:3]), nxt[0]) == want
    taken, _, nxt = _run(L, [9], p, d, tok, u, parent, max_rows=0)
    assert taken[0] == 0 and nxt[0] == -1


def test_rows_past_two_to_the_31_elements(L):
    """A row whose offset exceeds 32 bits."""
    V, N = 2 ** 22, 520
    p = torch.zeros(N, V, device=DEV)
    rng = np.random.default_rng(1)
    w = _soft(rng, 2, V, 1.0)
    p[N - 2:] = torch.from_numpy(w)
    i32 = lambda a: torch.tensor(a, dtype=torch.int32, device=DEV)  # noqa: E731
    tok = np.zeros(N, np.int32)
    tok[N - 1] = int(np.argmax(w[0]))
    for ua in (0.0, 0.9):
        u = np.full(N, 0.37, np.float32)
        u[N - 1] = ua
        taken, nxt, path = i32([7]), i32([7]), i32([7] * N)
        ws = torch.empty(L.qe_verify_workspace_bytes(1, V), dtype=torch.uint8, device=DEV)
        L.qe_verify_drafts(p, i32([N - 2, N]), i32(tok), torch.from_numpy(u).to(DEV), taken, path, nxt, ws, max_rows=2)
        want, token = C.verify(w, tok[N - 2:], u[N - 2:])
        assert int(taken) == len(want) and int(nxt) == token
        assert path[N - 2:].tolist() == want + [-1] * (2 - len(want))
        assert bool((path[:N - 2] == 7).all())
