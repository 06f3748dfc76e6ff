"""GPU parity of the rotary positions and of the append to the paged cache.

Cosines and sines are float64 values rounded to float32 (2^-24 relative), each product and the sum round once more: a
turned float32 channel is within 3.5 * 2^-24 (|x1| + |x2|) scale of the definition, a bf16 one half a step (2^-8
relative) further.  The 8-bit codes are those of the library's own quantization of the turned float32 heads, bit for bit.
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
def L():
    from quantized_linear_moe_amd import libqe
    return libqe


def _rope(L, rot, pairs=False, sections=None, scale=1.0, base=1e4):
    f, _ = C.freqs(rot, base)
    return L.make_rope(torch.from_numpy(f).to(DEV), pairs=pairs, sections=sections, scale=scale), f


def _check_turned(y, x, pos, f, pairs, sections, scale, dtype):
    want = C.rope(x.float().cpu().numpy(), pos.cpu().numpy(), f, pairs, sections, scale)
    xa = np.abs(x.float().cpu().numpy().astype(np.float64))
    half = len(f)
    reach = np.zeros_like(xa)
    a, b = (slice(0, 2 * half, 2), slice(1, 2 * half, 2)) if pairs else (slice(0, half), slice(half, 2 * half))
    reach[..., a] = reach[..., b] = xa[..., a] + xa[..., b]
    tol = 3.5 * 2.0 ** -24 * reach * scale
    if dtype == BF:
        tol = tol * (1 + 2.0 ** -8) + 2.0 ** -8 * np.abs(want)
    got = y.float().cpu().numpy().astype(np.float64)
    if dtype != BF or x.dtype == BF:  # channels past the rotation are copies
        assert np.array_equal(got[..., 2 * half:], x.float().cpu().numpy()[..., 2 * half:])
    assert np.all(np.abs(got - want) <= tol), float((np.abs(got - want) - tol).max())


@pytest.mark.parametrize("xd,yd", [(BF, BF), (torch.float32, torch.float32), (torch.float32, BF), (BF, torch.float32)])
@pytest.mark.parametrize("T,heads,hd,rot", [(1, 1, 16, 16), (1, 12, 128, 128), (3, 5, 64, 32), (37, 3, 80, 80),
                                            (130, 2, 96, 48), (9, 40, 256, 256), (17, 1, 256, 16), (5, 7, 112, 112)])
@pytest.mark.parametrize("pairs", [False, True])
def test_rope(L, T, heads, hd, rot, xd, yd, pairs):
    g = torch.Generator().manual_seed(T + hd)
    x = torch.randn(T, heads, hd, generator=g).to(xd).to(DEV)
    pos = torch.randint(0, 5000, (1, T), generator=g, dtype=torch.int32).to(DEV)
    rope, f = _rope(L, rot, pairs)
    y = torch.full((T + 1, heads, hd), 77.0, dtype=yd, device=DEV)
    L.qe_rope_apply(rope, pos, x, y[:T])
    torch.cuda.synchronize()
    assert bool((y[T] == 77).all())
    _check_turned(y[:T], x, pos, f, pairs, None, 1.0, yd)


@pytest.mark.parametrize("sections", [(16, 24, 24), (0, 0, 64), (64, 0, 0), (1, 62, 1), (0, 64, 0)])
def test_rope_sections(L, sections):
    T = 50
    g = torch.Generator().manual_seed(1)
    x = torch.randn(T, 4, 128, generator=g).to(DEV)
    pos = torch.randint(0, 4000, (3, T), generator=g, dtype=torch.int32).to(DEV)
    rope, f = _rope(L, 128, sections=sections, scale=1.25, base=1e6)
    y = torch.empty_like(x)
    L.qe_rope_apply(rope, pos, x, y)
    _check_turned(y, x, pos, f, False, sections, 1.25, torch.float32)


def test_rope_far_positions(L):
    """Positions up to 2^31 - 1 and below zero: the angle's product is rounded once (2^-53), which moves it by at
    most 2^-22 at 2^31; positions up to 2^20 keep the ordinary bound."""
    pos = torch.tensor([[0, 1, 2 ** 20, 999999, -5, 2 ** 20 - 1]], dtype=torch.int32, device=DEV)
    x = torch.randn(6, 2, 64, generator=torch.Generator().manual_seed(2)).to(DEV)
    rope, f = _rope(L, 64)
    y = torch.empty_like(x)
    L.qe_rope_apply(rope, pos, x, y)
    _check_turned(y, x, pos, f, False, None, 1.0, torch.float32)
    pos = torch.tensor([[2 ** 31 - 1, -2 ** 31]], dtype=torch.int32, device=DEV)
    y = torch.empty_like(x[:2])
    L.qe_rope_apply(rope, pos, x[:2], y)
    want = C.rope(x[:2].cpu().numpy(), pos.cpu().numpy(), f)
    assert np.abs(y.cpu().numpy() - want).max() <= (3.5 * 2.0 ** -24 + 2 * 2.0 ** -22) * 2 * float(x.abs().max())


@pytest.mark.parametrize("pairs", [False, True])
def test_rope_in_place_and_strided(L, pairs):
    """q and k side by side in one row, turned in place; the v part and the gap behind it are kept."""
    T, heads, hd = 41, 6, 64
    buf = torch.randn(T, (heads + 2) * hd + 24, generator=torch.Generator().manual_seed(4)).to(BF).to(DEV)
    was = buf.clone()
    part = buf[:, 8:8 + heads * hd].unflatten(1, (heads, hd))
    pos = torch.arange(T, dtype=torch.int32, device=DEV)
    rope, f = _rope(L, 64, pairs)
    L.qe_rope_apply(rope, pos, part, part)
    torch.cuda.synchronize()
    _check_turned(part, was[:, 8:8 + heads * hd].unflatten(1, (heads, hd)), pos[None], f, pairs, None, 1.0, BF)
    assert torch.equal(buf[:, :8], was[:, :8]) and torch.equal(buf[:, 8 + heads * hd:], was[:, 8 + heads * hd:])


def _new_cache(L, pages, kv, page, hd, i8):
    if not i8:
        k, v = (torch.full((pages, kv, page, hd), 7.0, dtype=BF, device=DEV) for _ in range(2))
        return L.make_cache(k, v), (k, v, None, None)
    k, v = (torch.full((pages, kv, page, hd), 7, dtype=torch.int8, device=DEV) for _ in range(2))
    ks, vs = (torch.full((pages, kv, page), 7.0, device=DEV) for _ in range(2))
    return L.make_cache(k, v, ks, vs), (k, v, ks, vs)


@pytest.mark.parametrize("i8", [False, True])
@pytest.mark.parametrize("xd", [BF, torch.float32])
@pytest.mark.parametrize("T,kv,heads,hd,rot,page", [(1, 2, 12, 128, 128, 16), (33, 1, 0, 64, 64, 8), (70, 3, 3, 80, 48, 32),
                                                    (20, 8, 64, 128, 128, 1), (130, 2, 2, 256, 256, 1024),
                                                    (45, 4, 28, 96, 96, 64), (3, 1, 1, 16, 16, 2)])
def test_append(L, T, kv, heads, hd, rot, page, xd, i8):
    g = torch.Generator().manual_seed(T * 3 + hd)
    k, v = (torch.randn(T, kv, hd, generator=g).to(xd).to(DEV) for _ in range(2))
    k[:, :, 0] *= 9
    v[0] = 0  # a head of zeros
    q = torch.randn(T, heads, hd, generator=g).to(xd).to(DEV) if heads else None
    pos = torch.randint(0, 3000, (1, T), generator=g, dtype=torch.int32).to(DEV)
    pages = (T + page - 1) // page + 2
    slot = torch.randperm(pages * page, generator=g)[:T].to(torch.int32)
    if T > 2:
        slot[1], slot[2] = -1, pages * page  # padding, and a place past the cache
    slot = slot.to(DEV)
    rope, f = _rope(L, rot)
    cache, (ck, cv, ks, vs) = _new_cache(L, pages, kv, page, hd, i8)
    q_out = torch.empty(T, heads, hd, dtype=BF, device=DEV) if heads else None
    L.qe_kv_append(cache, k, v, slot, rope=rope, pos=pos, q=q, q_out=q_out)
    torch.cuda.synchronize()
    if heads:
        _check_turned(q_out, q, pos, f, False, None, 1.0, BF)
    at = torch.nonzero((slot >= 0) & (slot < pages * page))[:, 0]
    where = slot[at].long()
    turned = torch.empty(T, kv, hd, device=DEV)  # the keys as the library turns them, in float32
    L.qe_rope_apply(rope, pos, k, turned)
    for x, c, s in ((turned, ck, ks), (v.float(), cv, vs)):
        got = c[where // page, :, where % page]
        if i8:
            codes, scales = O.quant_act(x[at].cpu().numpy().reshape(-1, hd), None, 8)
            assert np.array_equal(got.cpu().numpy().reshape(-1, hd), codes)
            assert np.array_equal(s[where // page, :, where % page].cpu().numpy().reshape(-1), scales)
        else:
            assert torch.equal(got, x[at].to(BF))
        rest = torch.ones(pages * page, dtype=torch.bool, device=DEV)
        rest[where] = False
        other = c.transpose(1, 2).reshape(pages * page, kv, hd)[rest]
        assert bool((other == 7).all()), "a place that no token names was written"
        if i8:
            assert bool((s.transpose(1, 2).reshape(pages * page, kv)[rest] == 7).all())


def test_append_without_rotation_and_strided(L):
    T, kv, heads, hd = 19, 2, 4, 64
    rows = torch.randn(T, (heads + 2 * kv) * hd + 8, generator=torch.Generator().manual_seed(6)).to(BF).to(DEV)
    q = rows[:, :heads * hd].unflatten(1, (heads, hd))
    k = rows[:, heads * hd:(heads + kv) * hd].unflatten(1, (kv, hd))
    v = rows[:, (heads + kv) * hd:(heads + 2 * kv) * hd].unflatten(1, (kv, hd))
    cache, (ck, cv, _, _) = _new_cache(L, 3, kv, 8, hd, False)
    slot = torch.arange(T, dtype=torch.int32, device=DEV)
    q_out = torch.empty(T, heads, hd, device=DEV)
    L.qe_kv_append(cache, k, v, slot, q=q, q_out=q_out)
    s = slot.long()
    assert torch.equal(ck[s // 8, :, s % 8], k) and torch.equal(cv[s // 8, :, s % 8], v)
    assert torch.equal(q_out, q.float())


def test_append_past_two_to_the_31_elements(L):
    """Places whose offset in the cache exceeds 32 bits, in elements and in bytes."""
    kv, hd, page = 2, 256, 1024
    pages = 4200  # 2.2 * 10^9 elements
    k = torch.empty(pages, kv, page, hd, dtype=torch.int8, device=DEV)
    v = torch.empty_like(k)
    ks, vs = (torch.zeros(pages, kv, page, device=DEV) for _ in range(2))
    cache = L.make_cache(k, v, ks, vs)
    T = 4
    x = torch.randn(T, kv, hd, generator=torch.Generator().manual_seed(8)).to(DEV)
    slot = torch.tensor([pages * page - 1, 4100 * page, 4199 * page + 5, 0], dtype=torch.int32, device=DEV)
    L.qe_kv_append(cache, x, x, slot)
    codes, scales = O.quant_act(x.cpu().numpy().reshape(-1, hd), None, 8)
    s = slot.long()
    for c, sc in ((k, ks), (v, vs)):
        assert np.array_equal(c[s // page, :, s % page].cpu().numpy().reshape(-1, hd), codes)
        assert np.array_equal(sc[s // page, :, s % page].cpu().numpy().reshape(-1), scales)
