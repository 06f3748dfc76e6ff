"""Attention past the bounds that a call names, over long pieces, and of values near the end of their range; against the
definition in float64, with the bound of test_gpu_attention.py."""

import numpy as np
import pytest
import torch

from oracle import qe_cache_oracle as C
from test_gpu_attention import BF, DEV, Batch, _forest

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def L():
    from quantized_linear_moe_amd import libqe
    return libqe


def _i32(a):
    return torch.tensor(a, dtype=torch.int32, device=DEV)


def _first(cut):
    """Only the first cut keys are there."""
    def seen_of(s, seen):
        seen = seen.copy()
        seen[:, cut:] = False
        return seen
    return seen_of


@pytest.mark.parametrize("i8", [False, True])
@pytest.mark.parametrize("tree", [False, True])
@pytest.mark.parametrize("n,length,cut", [(2, 100, 98), (2, 100, 99), (3, 64, 32), (7, 700, 640), (10, 100, 90), (60, 60, 16),
                                          (60, 300, 256), (40, 1000, 976), (33, 100, 48)])
def test_keys_past_the_bounds_are_left_out(L, n, length, cut, tree, i8):
    """The new tokens are the last of kv_len keys whatever max_kv and the page table keep of them."""
    lens = [(n, length), (n, length)]
    bits = _forest(np.random.default_rng(n + cut), lens) if tree else None
    b = Batch(L, lens, 8, 2, 64, 16, i8, tree=bits, seed=n, tail=1)
    b.check(b.run(L, max_kv=cut), seen_of=_first(cut))
    cut -= cut % 16
    b.pages_dev = b.pages[:, :cut // 16].contiguous().to(DEV)
    b.check(b.run(L), seen_of=_first(cut))


@pytest.mark.parametrize("n", [1, 3, 50])
def test_lengths_far_past_the_bounds(L, n):
    """Every key that there is lies before the new tokens."""
    for tree in (None, _forest(np.random.default_rng(n), [(n, 112)])):
        b = Batch(L, [(n, 112)], 4, 2, 64, 16, tree=tree, seed=n)
        for length in (2 ** 31 - 1, 2 ** 30, 112 + n):
            b.kv_len = _i32([length])
            for max_kv in (112, 4000, 2 ** 30):
                b.check(b.run(L, max_kv=max_kv), seen_of=lambda s, seen: np.ones_like(seen))


@pytest.mark.parametrize("i8", [False, True])
@pytest.mark.parametrize("n", [2, 5, 40])
def test_infinities_behind_the_tokens_that_max_q_keeps(L, n, i8):
    """The keys of the tokens that are left out stay unseen, whatever they hold."""
    for keep in (1, n - 1):
        b = Batch(L, [(n, 90)], 4, 2, 64, 16, i8, seed=n)
        full = b.run(L)
        for j in range(90 - n + keep, 90):
            page, place = int(b.pages[0, j // 16]), j % 16
            for x, value in zip((b.ks, b.vs) if i8 else (b.k, b.v), (float("nan"), float("inf"))):
                x[page, :, place] = value
        for t, x in zip(b.tensors, (b.k, b.v, b.ks, b.vs)):
            if x is not None:
                t.copy_(x)
        out = b.run(L, max_q=keep)
        assert bool((out[keep:] == 77).all()) and bool(torch.isfinite(out[:keep]).all())
        # the same keys; another launch may sum them in another order, each within its bound of 2^-6 sum p |v|
        top = 127 * float(b.vs[torch.isfinite(b.vs)].max()) if i8 else float(b.v[torch.isfinite(b.v)].abs().max())
        assert float((out[:keep].float() - full[:keep].float()).abs().max()) <= 2.0 ** -5 * top


@pytest.mark.parametrize("i8", [False, True])
@pytest.mark.parametrize("n,length", [(1, 2), (1, 300), (1, 3000), (3, 40), (40, 300), (33, 2000)])
def test_values_near_the_end_of_their_range(L, n, length, i8):
    """The sums of weighted values stay finite where the rows are: equal scores, and scores that grow along the keys."""
    for steep in (0.0, 1.0):
        b = Batch(L, [(n, length)], 4, 2, 64, 16, i8, seed=length)
        j = torch.arange(length)
        p, o = b.pages[0].long()[j // 16], j % 16
        if i8:
            b.vs[p, :, o] = 2.2e36
            b.v.abs_()
            b.ks[p, :, o] = (steep * j / length / 127)[:, None].expand(length, 2).contiguous()
            b.k.fill_(127)
        else:
            b.v[p, :, o] = (2.9e38 * (1 - torch.rand(length, 2, 64, generator=torch.Generator().manual_seed(n)) / 8)).to(BF)
            b.k[p, :, o] = (steep * j / length)[:, None, None].expand(length, 2, 64).to(BF)
        b.q_rows.copy_(b.q_rows.abs())
        for t, x in zip(b.tensors, (b.k, b.v, b.ks, b.vs)):
            if x is not None:
                t.copy_(x)
        b.check(b.run(L))


@pytest.mark.parametrize("i8", [False, True])
@pytest.mark.parametrize("n,length", [(1, 300), (1, 3000), (40, 2000)])
def test_small_values(L, n, length, i8):
    """Weights are at least 2^-c of their row's sum where they count (c = 8 + the bits of the length).  What that adds to the
    bound, after the division: bf16 products below 2^-126 are rounded to steps of 2^-149, 2^(c - 149) a key; with an 8-bit
    cache a weight times its scale may vanish below 2^-126, 127 * 2^(c - 126) a key."""
    b = Batch(L, [(n, length)], 4, 2, 64, 16, i8, seed=length)
    if i8:
        b.vs.mul_(1e-24)
    else:
        b.v.copy_((b.v.float() * 1e-34).to(BF))
    for t, x in zip(b.tensors, (b.k, b.v, b.ks, b.vs)):
        if x is not None:
            t.copy_(x)
    out = b.run(L).float().cpu().numpy().astype(np.float64)
    seen = C.sees(n, length - n, length)
    o, A, reach = C.attention(b.q.float().cpu().numpy(), *b.keys_of(0, length), seen, 64 ** -0.5)
    count = seen.sum(1)[:, None, None]
    c = 8 + length.bit_length()
    d = 64 ** -0.5 * reach * (65 * 2.0 ** -23 + 8 * 2.0 ** -24) * 2
    tol = 2.0 ** -8 * np.abs(o) + (1 + 2.0 ** -8) * A * (2 * 2.0 ** -8 + 2 * np.expm1(d) + 2.0 ** -20 + 2 * count * 2.0 ** -23)
    tol = tol + count * (127 * 2.0 ** (c - 126) if i8 else 2.0 ** (c - 149))
    assert np.all(np.abs(out - o) <= tol)
    # the bound says something: at most 3000 * 2^(20 - 149) = 4.4e-36 beside A near 0.8e-34, with the 2^-7 of above 0.067
    assert np.median(tol / A) < 0.1


def _long(L, form, i8, whole, seed, hd=64, tree=False):
    """Two long sequences; whole: among so many short ones that keys are not divided."""
    n, short = (1, 400) if form == "few" else (40, 80)
    lens = [(n, 2300)] + [(1, 1 + s % 30) for s in range(short if whole else 0)] + [(n, 2049)]
    bits = _forest(np.random.default_rng(seed), lens) if tree else None
    b = Batch(L, lens, 8, 8, hd, 16, i8, tree=bits, seed=seed, tail=1)
    pieces = L.qe_attention_workspace_bytes(b.cache, 8, b.T + 1, len(lens), n, 2300) > 0
    assert pieces != whole
    return b


@pytest.mark.parametrize("i8", [False, True])
@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("form,tree", [("few", False), ("rows", False), ("rows", True)])
@pytest.mark.parametrize("whole", [True, False])
def test_long_pieces(L, whole, form, tree, hd, i8):
    """More than 128 pages of 16 in one piece, and pages outside the cache among the first 64 and far behind."""
    b = _long(L, form, i8, whole, 3, hd, tree)
    b.check(b.run(L))
    bad = [5, 63, 64, 70, 127, 128, 140]
    pages = b.pages.clone()
    for i, p in enumerate(bad):
        pages[0, p] = (-1, b.k.shape[0], 2 ** 31 - 1, -2 ** 31)[i % 4]
    b.pages_dev = pages.to(DEV)

    def seen_of(s, seen):
        seen = seen.copy()
        for p in bad if s == 0 else []:
            seen[:, p * 16:(p + 1) * 16] = False
        return seen
    b.check(b.run(L), seen_of=seen_of)


@pytest.mark.parametrize("i8", [False, True])
@pytest.mark.parametrize("form", ["few", "rows"])
@pytest.mark.parametrize("whole", [True, False])
def test_keys_at_borders_count_once(L, whole, form, i8):
    """Nearly all weight on keys beside the borders of tiles, waves, pieces and windows of pages, each a like share: one
    left out or taken twice moves the row by a multiple of the bound."""
    b = _long(L, form, i8, whole, 4)
    for s, (n, length) in ((0, b.lens[0]), (len(b.lens) - 1, b.lens[-1])):
        j = torch.arange(length)
        p, o = b.pages[s].long()[j // 16], j % 16
        at = torch.tensor(sorted({0, 31, 32, 63, 64, 127, 128, 255, 256, 511, 512, 1023, 1024, 1151, 1152, 2047, 2048,
                                  length - 41, length - 1}))
        f = torch.full((length,), 1e-3)
        f[at] = 3.0
        if i8:
            b.k[p, :, o] = 127
            b.ks[p, :, o] = (f / 127)[:, None].expand(length, 8).contiguous()
        else:
            b.k[p, :, o] = f[:, None, None].to(BF).expand(length, 8, 64)
    b.q_rows.copy_(b.q_rows.abs())
    for t, x in zip(b.tensors, (b.k, b.v, b.ks, b.vs)):
        if x is not None:
            t.copy_(x)
    b.check(b.run(L))
