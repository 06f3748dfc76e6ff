"""GPU parity of the attention over the paged cache with the definition in float64.

Bound of an output channel, with p the exact weights, A = sum_j p_j |v_j| and n the visible keys:
  scores     each of hd + 1 float32 additions of exact products is off by at most a step (2^-23) of the sum of
             magnitudes, the scaling and the difference to the maximum by a few 2^-24 of the score's reach; a score's
             error d multiplies its weight by e^d
  weights    bf16: half a step, 2^-8 relative; the sum they are divided by is made of the same rounded weights or of
             unrounded ones: 2 * 2^-8 A in all; exp2 and the factors of the running maximum: 2^-20
  sums       n additions each of the weights and of the products: 2 n 2^-23 A
  output     half a step of bf16, 2^-8 |o|
"""

import numpy as np
import pytest
import torch

from oracle import qe_cache_oracle as C

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF = torch.bfloat16


@pytest.fixture(scope="module")
def L():
    from quantized_linear_moe_amd import libqe
    return libqe


class Batch:
    """Sequences with (new tokens, keys) over a cache whose unlisted places hold NaN (8-bit: NaN scales)."""

    def __init__(self, L, lens, heads, kv, hd, page, i8=False, tree=None, seed=0, tail=0, spare=3, q_pad=0):
        g = torch.Generator().manual_seed(seed)
        self.lens, self.heads, self.kv, self.hd, self.page, self.i8 = lens, heads, kv, hd, page, i8
        need = [(k + page - 1) // page for _, k in lens]
        pool, self.width = sum(need) + spare, max(need + [1])
        order = torch.randperm(pool, generator=g).to(torch.int32)
        self.pages = torch.full((len(lens), self.width), 2 ** 31 - 1, dtype=torch.int32)
        at = 0
        for s, n in enumerate(need):
            self.pages[s, :n] = order[at:at + n]
            at += n
        used = torch.zeros(pool, page, dtype=torch.bool)
        for s, (_, n) in enumerate(lens):
            j = torch.arange(n)
            used[self.pages[s].long()[j // page], j % page] = True
        keep = used[:, None, :, None].expand(pool, kv, page, hd)
        if i8:
            self.k, self.v = (torch.randint(-127, 128, (pool, kv, page, hd), generator=g).to(torch.int8) for _ in range(2))
            self.ks, self.vs = (((0.5 + torch.rand(pool, kv, page, generator=g)) / 64).masked_fill(
                ~used[:, None].expand(pool, kv, page), float("nan")) for _ in range(2))
        else:
            self.k, self.v = (torch.randn(pool, kv, page, hd, generator=g).to(BF).masked_fill(~keep, float("nan"))
                              for _ in range(2))
            self.ks = self.vs = None
        self.T = sum(n for n, _ in lens)
        self.tail = tail
        wide = torch.randn(self.T + tail, heads * hd + q_pad, generator=g) * 1.5
        self.q_rows = wide.to(BF).to(DEV)
        self.q = self.q_rows[:, :heads * hd].unflatten(1, (heads, hd))
        starts = np.cumsum([0] + [n for n, _ in lens])
        self.starts = starts
        i32 = lambda a: torch.tensor(np.asarray(a), dtype=torch.int32, device=DEV)  # noqa: E731
        self.q_start, self.kv_len = i32(starts), i32([k for _, k in lens])
        self.tree = tree
        self.tree_dev = None
        if tree is not None:
            self.tree_dev = torch.from_numpy(np.concatenate([tree, np.full((tail, tree.shape[1]), 2 ** 32 - 1, np.uint32)])
                                             .view(np.int32)).to(DEV)
        dev = lambda t: None if t is None else t.to(DEV)  # noqa: E731
        self.tensors = [dev(t) for t in (self.k, self.v, self.ks, self.vs)]
        self.cache = L.make_cache(*self.tensors)
        self.pages_dev = self.pages.to(DEV)
        self.max_q, self.max_kv = max([n for n, _ in lens] + [0]), max([k for _, k in lens] + [0])

    def workspace(self, L, max_q=None, max_kv=None):
        n = L.qe_attention_workspace_bytes(self.cache, self.heads, self.T + self.tail, len(self.lens),
                                           self.max_q if max_q is None else max_q, self.max_kv if max_kv is None else max_kv)
        return torch.full((max(n, 16),), 255, dtype=torch.uint8, device=DEV)

    def run(self, L, scale=None, out=None, ws=None, max_q=None, max_kv=None, stream=None):
        if out is None:
            out = torch.full((self.T + self.tail, self.heads, self.hd), 77.0, dtype=BF, device=DEV)
        L.qe_attention(self.cache, self.q, self.q_start, self.kv_len, self.pages_dev,
                       self.max_q if max_q is None else max_q, self.max_kv if max_kv is None else max_kv, out,
                       self.workspace(L, max_q, max_kv) if ws is None else ws, tree=self.tree_dev, scale=scale, stream=stream)
        return out

    def keys_of(self, s, length):
        j = torch.arange(length)
        p, o = self.pages[s].long()[j // self.page], j % self.page
        out = []
        for x, sc in ((self.k, self.ks), (self.v, self.vs)):
            a = x[p, :, o].double()
            out.append((a * sc[p, :, o].double()[..., None] if self.i8 else a).numpy())
        return out

    def check(self, out, scale=None, seen_of=None):
        scale = self.hd ** -0.5 if scale is None else scale
        got = out.float().cpu().numpy().astype(np.float64)
        q = self.q.float().cpu().numpy()
        for s, (n, length) in enumerate(self.lens):
            a = self.starts[s]
            if n == 0:
                continue
            K, V = self.keys_of(s, length)
            seen = C.sees(n, length - n, length, None if self.tree is None else self.tree[a:a + n])
            if seen_of:
                seen = seen_of(s, seen)
            o, A, reach = C.attention(q[a:a + n], K, V, seen, scale)
            d = scale * reach * ((self.hd + 1) * 2.0 ** -23 + 8 * 2.0 ** -24) * 2  # of a score and of the maximum's
            count = seen.sum(1)[:, None, None]
            tol = 2.0 ** -8 * np.abs(o) + (1 + 2.0 ** -8) * A * (2 * 2.0 ** -8 + 2 * np.expm1(d) + 2.0 ** -20 +
                                                                 2 * count * 2.0 ** -23)
            err = np.abs(got[a:a + n] - o)
            assert np.all(err <= tol), f"sequence {s}: {float((err - tol).max())}"
            assert np.all(got[a:a + n][~seen.any(1)] == 0)
        if self.tail:
            assert np.all(got[self.T:] == 77), "rows behind the last sequence were written"


def _forest(rng, lens, words=None, blank=0.0):
    """Ancestor bits of random trees; blank: the share of tokens that see none of the new ones."""
    words = words or max(1, (max(n for n, _ in lens) + 31) // 32)
    rows = []
    for n, _ in lens:
        m = np.zeros((n, words), np.uint32)
        for i in range(n):
            p = rng.integers(-1, i) if i else -1
            if p >= 0:
                m[i] = m[p]
            if i < 32 * words:
                m[i, i // 32] |= np.uint32(1 << (i % 32))
            if rng.random() < blank:
                m[i] = 0
        rows.append(m)
    return np.concatenate(rows)


LAYOUTS = [(1, 1), (4, 4), (8, 2), (6, 1), (14, 2), (8, 1)]


@pytest.mark.parametrize("i8", [False, True])
@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("heads,kv", LAYOUTS)
@pytest.mark.parametrize("length", [1, 2, 31, 32, 33, 130, 257, 1000])
def test_single_tokens(L, length, heads, kv, hd, i8):
    b = Batch(L, [(1, length)], heads, kv, hd, 16, i8, seed=length + heads)
    b.check(b.run(L))


@pytest.mark.parametrize("i8", [False, True])
@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("page", [1, 2, 8, 16, 64, 256, 1024])
def test_page_sizes(L, page, hd, i8):
    b = Batch(L, [(1, 300), (1, 7), (1, 65)], 8, 2, hd, page, i8, seed=page)
    b.check(b.run(L))
    b = Batch(L, [(40, 300), (3, 7), (33, 65)], 8, 2, hd, page, i8, seed=page + 1, tail=2)
    b.check(b.run(L))


@pytest.mark.parametrize("i8", [False, True])
@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("heads,kv", LAYOUTS)
@pytest.mark.parametrize("n,length", [(2, 2), (5, 40), (32, 32), (33, 97), (64, 64), (65, 200), (150, 150)])
def test_text(L, n, length, heads, kv, hd, i8):
    b = Batch(L, [(n, length)], heads, kv, hd, 16, i8, seed=n + heads, tail=1)
    b.check(b.run(L))


@pytest.mark.parametrize("i8", [False, True])
@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("heads,kv", [(4, 4), (14, 2)])
@pytest.mark.parametrize("blank", [0.0, 0.4])
@pytest.mark.parametrize("lens", [[(2, 3)], [(7, 7)], [(33, 50)], [(48, 300), (1, 200), (17, 17)], [(70, 129), (64, 1000)]])
def test_trees(L, lens, blank, heads, kv, hd, i8):
    rng = np.random.default_rng(len(lens) + lens[0][0])
    b = Batch(L, lens, heads, kv, hd, 16, i8, tree=_forest(rng, lens, blank=blank), seed=5, tail=3)
    b.check(b.run(L))


def test_tokens_that_see_nothing(L):
    """Whole trees of blank rows without context (rows of zeros), and words fewer than the tree's tokens."""
    for n in (3, 60):
        lens = [(n, n), (n, n + 5)]
        tree = _forest(np.random.default_rng(1), lens, blank=1.0)
        b = Batch(L, lens, 4, 2, 64, 8, tree=tree)
        out = b.run(L)
        b.check(out)
        assert bool((out[:n] == 0).all())
    lens = [(50, 90)]
    b = Batch(L, lens, 4, 2, 64, 8, tree=_forest(np.random.default_rng(2), lens, words=1))
    b.check(b.run(L))


@pytest.mark.parametrize("i8", [False, True])
@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("tree", [False, True])
@pytest.mark.parametrize("lens", [[(3, 3)], [(6, 200)], [(20, 25), (9, 140)], [(70, 90), (41, 700)]])
def test_infinities_and_nan_stay_with_the_rows_that_see_them(L, lens, tree, hd, i8):
    """A later token's key and value, or another branch's, may be anything: the rows that do not see it keep theirs."""
    tree = _forest(np.random.default_rng(7), lens, blank=0.2) if tree else None
    b = Batch(L, lens, 4, 2, hd, 8, i8, tree=tree, seed=11)
    for s, (n, length) in enumerate(lens):
        for token, of, channel, value in ((n // 2, 1, 3, float("inf")), (n // 2 + 1, 1, 5, float("nan")),
                                          (n - 1, 0, 7, float("nan")), (n - 1, 1, 9, float("-inf"))):
            j = length - n + token
            page, place = int(b.pages[s, j // 8]), j % 8
            if i8:
                (b.ks, b.vs)[of][page, :, place] = value
            else:
                (b.k, b.v)[of][page, :, place, channel] = value
    for t, x in zip(b.tensors, (b.k, b.v, b.ks, b.vs)):
        if x is not None:
            t.copy_(x)
    out = b.run(L)
    got = out.float().cpu().numpy().astype(np.float64)
    finite = 0
    for s, (n, length) in enumerate(lens):
        a = b.starts[s]
        seen = C.sees(n, length - n, length, None if tree is None else tree[a:a + n])
        with np.errstate(invalid="ignore"):
            o = C.attention(b.q[a:a + n].float().cpu().numpy(), *b.keys_of(s, length), seen, hd ** -0.5)[0]
        ok = np.isfinite(o)
        finite += ok.sum()
        assert np.array_equal(np.isfinite(got[a:a + n]), ok)
        got[a:a + n][~ok] = 0
    assert finite > 0
    # what is finite, against a cache in which those places are zeros
    for x in (b.k, b.v, b.ks, b.vs):
        if x is not None and x.dtype != torch.int8:
            x.nan_to_num_(0.0, 0.0, 0.0)
    for s, (n, length) in enumerate(lens):
        a = b.starts[s]
        seen = C.sees(n, length - n, length, None if tree is None else tree[a:a + n])
        o, A, reach = C.attention(b.q[a:a + n].float().cpu().numpy(), *b.keys_of(s, length), seen, hd ** -0.5)
        d = hd ** -0.5 * reach * ((hd + 1) * 2.0 ** -23 + 8 * 2.0 ** -24) * 2
        tol = 2.0 ** -8 * np.abs(o) + (1 + 2.0 ** -8) * A * (2 * 2.0 ** -8 + 2 * np.expm1(d) + 2.0 ** -20 +
                                                             2 * seen.sum(1)[:, None, None] * 2.0 ** -23)
        ok = np.isfinite(out.float().cpu().numpy()[a:a + n])
        assert np.all((np.abs(got[a:a + n] - o) <= tol)[ok])


def test_empty_and_short_sequences(L):
    """No new tokens, no keys at all, fewer keys than new tokens (the first ones' are missing)."""
    for n in (1, 5, 40):
        b = Batch(L, [(0, 10), (n, 0), (n, n - 1), (0, 0), (n, 80)], 8, 2, 64, 16, tail=2, seed=n)
        out = b.run(L)
        b.check(out)
        assert bool((out[:n] == 0).all())  # the sequence without keys
        tree = _forest(np.random.default_rng(n), b.lens)
        b = Batch(L, b.lens, 8, 2, 64, 16, tail=2, seed=n, tree=tree)
        b.check(b.run(L))


@pytest.mark.parametrize("i8", [False, True])
@pytest.mark.parametrize("n", [1, 30])
def test_pages_outside_the_cache(L, n, i8):
    """Their keys are not seen: the first page, one in the middle, and every page."""
    for bad in ([0], [3, 4], list(range(13))):
        b = Batch(L, [(n, 200), (n, 90)], 8, 2, 64, 16, i8, seed=3)
        pages = b.pages.clone()
        for i, p in enumerate(bad):
            pages[0, p] = (-1, b.k.shape[0], 2 ** 31 - 1, -2 ** 31)[i % 4]
        b.pages_dev = pages.to(DEV)

        def seen_of(s, seen):
            seen = seen.copy()
            if s == 0:
                for p in bad:
                    seen[:, p * 16:(p + 1) * 16] = False
            return seen
        b.check(b.run(L), seen_of=seen_of)


def test_lengths_are_cut(L):
    """Lengths past the page table, past max_kv and below zero; more new tokens than max_q; starts that run backwards."""
    b = Batch(L, [(2, 100)], 4, 2, 64, 16)
    full = b.run(L)
    b.kv_len = torch.tensor([2 ** 31 - 1], dtype=torch.int32, device=DEV)
    b.max_kv = 2 ** 30  # the table's 7 pages end the sequence at 112; its last places are NaN places
    b.run(L)
    b.kv_len = torch.tensor([-7], dtype=torch.int32, device=DEV)
    assert bool((b.run(L) == 0).all())
    b.kv_len = torch.tensor([100], dtype=torch.int32, device=DEV)
    assert torch.equal(b.run(L, max_kv=4096), full)
    b.q_start = torch.tensor([2, 0], dtype=torch.int32, device=DEV)
    assert bool((b.run(L) == 77).all())
    b.q_start = torch.tensor([0, 2 ** 31 - 1], dtype=torch.int32, device=DEV)  # cut to the two tokens
    assert torch.equal(b.run(L), full)
    b.q_start = torch.tensor([0, 2], dtype=torch.int32, device=DEV)
    out = b.run(L, max_q=1)
    assert torch.equal(out[0], full[0]) and bool((out[1] == 77).all())


@pytest.mark.parametrize("n", [1, 60])
def test_strides_and_scale(L, n):
    b = Batch(L, [(n, 150), (n, 70)], 8, 2, 128, 16, seed=9, q_pad=40)
    wide = torch.full((b.T, 8 * 128 + 16), 77.0, dtype=BF, device=DEV)
    out = wide[:, 8:8 + 8 * 128].unflatten(1, (8, 128))
    b.run(L, scale=0.31, out=out)
    b.check(out, scale=0.31)
    assert bool((wide[:, :8] == 77).all()) and bool((wide[:, 8 + 8 * 128:] == 77).all())


def test_steep_scores(L):
    """Scores of hundreds that grow along the sequence (the running maximum moves), fall, or sit on one key."""
    for kind in ("up", "down", "one"):
        for n in (1, 40):
            b = Batch(L, [(n, 400)], 4, 2, 64, 16, seed=2)
            j = torch.arange(400)
            f = {"up": j / 40.0, "down": (400 - j) / 40.0, "one": torch.where(j == 123, 12.0, 0.01)}[kind]
            p, o = b.pages[0].long()[j // 16], j % 16
            b.k[p, :, o] = (f[:, None, None] * torch.ones(64)).to(BF).expand(400, 2, 64)
            b.q_rows.copy_(b.q_rows.abs())
            b.tensors[0].copy_(b.k)
            b.check(b.run(L))


@pytest.mark.parametrize("i8", [False, True])
@pytest.mark.parametrize("n,tree", [(1, False), (4, False), (33, True), (100, False)])
def test_long_contexts_in_pieces(L, n, tree, i8):
    lens = [(n, 5000), (n, 129), (n, 2049)]
    bits = _forest(np.random.default_rng(n), lens) if tree else None
    b = Batch(L, lens, 8, 2, 128, 64, i8, tree=bits, seed=n, tail=1)
    assert L.qe_attention_workspace_bytes(b.cache, 8, b.T + 1, 3, n, 5000) > 0
    out = b.run(L)
    b.check(out)
    assert torch.equal(out, b.run(L))


@pytest.mark.parametrize("i8", [False, True])
@pytest.mark.parametrize("heads,kv", [(33, 1), (64, 1), (160, 2), (31, 1), (32, 1)])
def test_wide_groups(L, heads, kv, i8):
    """Groups of query heads around and past the 32 rows of a wave and the 128 of a tile."""
    for lens in ([(1, 77), (1, 300)], [(3, 50), (2, 129)]):
        b = Batch(L, lens, heads, kv, 64, 16, i8, seed=heads)
        b.check(b.run(L))


def test_bounds_above_the_lengths_change_nothing_visible(L):
    """A launch chosen for longer contexts and more tokens gives rows within the bound too."""
    for n in (1, 20):
        b = Batch(L, [(n, 90), (n, 33)], 8, 2, 64, 16, seed=n)
        for max_q, max_kv in ((n, 20000), (300, 90), (500, 100000)):
            b.check(b.run(L, max_q=max_q, max_kv=max_kv))


def test_long_prompt(L):
    """A prompt of many tiles (sampled rows against the definition)."""
    n = 1500
    b = Batch(L, [(n, n + 200)], 4, 1, 128, 32, seed=1)
    out = b.run(L).float().cpu().numpy().astype(np.float64)
    K, V = b.keys_of(0, n + 200)
    for i in (0, 1, 31, 32, 63, 64, 700, 1023, 1024, 1499):
        q = b.q[i:i + 1].float().cpu().numpy()
        o, A, reach = C.attention(q, K[:201 + i], V[:201 + i], np.ones((1, 201 + i), bool), 128 ** -0.5)
        d = 128 ** -0.5 * reach * (137 * 2.0 ** -23) * 2
        tol = 2.0 ** -8 * np.abs(o) + 1.01 * A * (2 * 2.0 ** -8 + 2 * np.expm1(d) + 2.0 ** -20 + 2 * (201 + i) * 2.0 ** -23)
        assert np.all(np.abs(out[i:i + 1] - o) <= tol)


def test_cache_past_two_to_the_31_elements(L):
    """Pages at the far end of a cache whose offsets exceed 32 bits."""
    kv, hd, page, pages = 2, 128, 1024, 8300  # 2.2 * 10^9 elements
    small = Batch(L, [(1, 2000), (40, 1500)], 8, kv, hd, page, seed=4)
    k, v = (torch.empty(pages, kv, page, hd, dtype=BF, device=DEV) for _ in range(2))
    shift = pages - small.k.shape[0]
    k[shift:], v[shift:] = small.tensors[0], small.tensors[1]
    want = small.run(L)
    small.cache = L.make_cache(k, v)
    small.pages_dev = (small.pages + shift).to(torch.int32).to(DEV)
    assert torch.equal(small.run(L), want)
    small.check(want)
