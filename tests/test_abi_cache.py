"""Argument checks of the rotary, cache, attention and verification entry points (no GPU needed: a refused call returns
before anything is enqueued), of their bindings, and the host frequencies."""

import ctypes

import numpy as np
import pytest
import torch

from oracle import qe_cache_oracle as C

P = 4096  # a 16-byte aligned address that no refused call reads


@pytest.fixture(scope="module")
def L():
    from quantized_linear_moe_amd import _libqe
    return _libqe


def _rope(L, **kw):
    a = dict(rot_dim=64, layout=0, n_pos=1, sections=(0, 0, 0), scale=1.0, inv_freq=P)
    a.update(kw)
    a["sections"] = (ctypes.c_int32 * 3)(*a["sections"])
    return L.qe_rope(*[a[k] for k in ("rot_dim", "layout", "n_pos", "sections", "scale", "inv_freq")])


def _cache(L, **kw):
    a = dict(n_kv_heads=2, head_dim=64, page_size=16, n_pages=8, dtype=L.QE_BF16, k=P, v=P, k_scale=None, v_scale=None)
    a.update(kw)
    return L.qe_kv_cache(*[a[k] for k in ("n_kv_heads", "head_dim", "page_size", "n_pages", "dtype", "k", "v", "k_scale",
                                          "v_scale")])


BAD_ROPES = [(dict(rot_dim=0), "INVALID_ARG"), (dict(rot_dim=-16), "INVALID_ARG"), (dict(rot_dim=80), "INVALID_ARG"),
             (dict(rot_dim=24), "UNSUPPORTED"), (dict(layout=2), "INVALID_ARG"), (dict(n_pos=2), "INVALID_ARG"),
             (dict(n_pos=3), "INVALID_ARG"), (dict(n_pos=3, sections=(16, 24, -8)), "INVALID_ARG"),
             (dict(n_pos=3, sections=(16, 8, 9)), "INVALID_ARG"),
             (dict(n_pos=3, sections=(2 ** 31 - 1, 2 ** 31 - 1, 34)), "INVALID_ARG"),
             (dict(scale=0.0), "INVALID_ARG"), (dict(scale=-1.0), "INVALID_ARG"),
             (dict(scale=float("nan")), "INVALID_ARG"), (dict(scale=float("inf")), "INVALID_ARG"),
             (dict(inv_freq=None), "INVALID_ARG"), (dict(inv_freq=P + 8), "ALIGNMENT")]

BAD_CACHES = [(dict(n_kv_heads=0), "INVALID_ARG"), (dict(n_kv_heads=5000), "UNSUPPORTED"), (dict(head_dim=0), "INVALID_ARG"),
              (dict(head_dim=72), "UNSUPPORTED"), (dict(head_dim=272), "UNSUPPORTED"), (dict(page_size=0), "INVALID_ARG"),
              (dict(page_size=24), "UNSUPPORTED"), (dict(page_size=2048), "UNSUPPORTED"), (dict(n_pages=0), "INVALID_ARG"),
              (dict(n_pages=2 ** 27), "UNSUPPORTED"), (dict(dtype=0), "INVALID_ARG"), (dict(dtype=3), "INVALID_ARG"),
              (dict(k=None), "INVALID_ARG"), (dict(v=None), "INVALID_ARG"), (dict(k=P + 4), "ALIGNMENT"),
              (dict(v=P + 8), "ALIGNMENT"), (dict(dtype=2), "INVALID_ARG"), (dict(k_scale=P, v_scale=P), "INVALID_ARG"),
              (dict(dtype=2, k_scale=P, v_scale=P + 4), "ALIGNMENT")]


def _refused(L, f, good, bad):
    for change, want in bad:
        args = list(good)
        for at, v in change.items():
            args[at] = v
        assert f(*args) == getattr(L, "QE_ERR_" + want), change


def test_rope_refusals(L):
    f, ref = L.raw_library().qe_rope_apply, ctypes.byref
    # rope pos x x_dtype x_stride T n_heads head_dim y y_dtype y_stride stream
    good = [ref(_rope(L)), P, P, 1, 256, 4, 4, 64, 2 * P, 1, 256, None]
    _refused(L, f, good, [({0: ref(_rope(L, **kw))}, want) for kw, want in BAD_ROPES])
    _refused(L, f, good, [
        ({0: None}, "INVALID_ARG"), ({1: None}, "INVALID_ARG"), ({2: None}, "INVALID_ARG"), ({8: None}, "INVALID_ARG"),
        ({3: 2}, "INVALID_ARG"), ({9: -1}, "INVALID_ARG"), ({4: 248}, "INVALID_ARG"), ({4: 260}, "ALIGNMENT"),
        ({10: 255}, "INVALID_ARG"), ({10: 257}, "ALIGNMENT"), ({5: -1}, "INVALID_ARG"), ({6: 0}, "INVALID_ARG"),
        ({5: 2 ** 31 - 1}, "UNSUPPORTED"), ({6: 4097}, "UNSUPPORTED"), ({7: 0}, "INVALID_ARG"), ({7: 72, 4: 288, 10: 288}, "UNSUPPORTED"),
        ({7: 272, 4: 2048, 10: 2048}, "UNSUPPORTED"), ({8: P, 10: 264}, "INVALID_ARG"), ({8: P, 9: 0}, "INVALID_ARG"),
        ({1: P + 2}, "ALIGNMENT"), ({2: P + 4}, "ALIGNMENT"), ({8: 2 * P + 8}, "ALIGNMENT")])
    args = list(good)
    args[1] = args[2] = args[8] = None
    args[5] = 0
    assert f(*args) == L.QE_OK


def test_append_refusals(L):
    f, ref = L.raw_library().qe_kv_append, ctypes.byref
    # cache k v x_dtype k_stride v_stride T slot rope pos q q_stride n_heads q_out q_out_dtype q_out_stride stream
    good = [ref(_cache(L)), P, P, 1, 128, 128, 4, P, ref(_rope(L)), P, P, 256, 4, 2 * P, 1, 256, None]
    _refused(L, f, good, [({0: ref(_cache(L, **kw))}, want) for kw, want in BAD_CACHES])
    _refused(L, f, good, [({8: ref(_rope(L, **kw))}, want) for kw, want in BAD_ROPES])
    _refused(L, f, good, [
        ({0: None}, "INVALID_ARG"), ({1: None}, "INVALID_ARG"), ({2: None}, "INVALID_ARG"), ({7: None}, "INVALID_ARG"),
        ({9: None}, "INVALID_ARG"), ({10: None}, "INVALID_ARG"), ({13: None}, "INVALID_ARG"), ({12: 0}, "INVALID_ARG"),
        ({12: -1}, "INVALID_ARG"), ({12: 5000}, "UNSUPPORTED"), ({3: 2}, "INVALID_ARG"), ({14: 2}, "INVALID_ARG"),
        ({4: 120}, "INVALID_ARG"), ({5: 130}, "ALIGNMENT"), ({6: -1}, "INVALID_ARG"), ({6: 2 ** 30}, "UNSUPPORTED"), ({11: 248}, "INVALID_ARG"),
        ({15: 258}, "ALIGNMENT"), ({13: P, 15: 512}, "INVALID_ARG"), ({13: P, 14: 0}, "INVALID_ARG"),
        ({1: P + 4}, "ALIGNMENT"), ({7: P + 2}, "ALIGNMENT"), ({9: P + 1}, "ALIGNMENT"), ({13: 2 * P + 4}, "ALIGNMENT")])
    args = list(good)
    for i in (1, 2, 7, 9, 10, 13):
        args[i] = None
    args[6] = 0
    assert f(*args) == L.QE_OK


def test_attention_refusals(L):
    lib, ref = L.raw_library(), ctypes.byref
    f = lib.qe_attention
    c = _cache(L)
    need = lib.qe_attention_workspace_bytes(ref(c), 4, 8, 2, 4, 4096)
    assert need > 0
    # cache q q_stride T n_heads q_start kv_len pages n_seq max_pages max_q max_kv tree words scale out out_stride ws bytes
    good = [ref(c), P, 256, 8, 4, P, P, P, 2, 256, 4, 4096, None, 0, 0.125, 2 * P, 256, P, need, None]
    _refused(L, f, good, [({0: ref(_cache(L, **kw))}, want) for kw, want in BAD_CACHES])
    _refused(L, f, good, [
        ({0: None}, "INVALID_ARG"), ({0: ref(_cache(L, head_dim=96)), 2: 384, 16: 384}, "UNSUPPORTED"),
        ({1: None}, "INVALID_ARG"), ({5: None}, "INVALID_ARG"), ({6: None}, "INVALID_ARG"), ({7: None}, "INVALID_ARG"),
        ({15: None}, "INVALID_ARG"), ({15: P}, "INVALID_ARG"), ({2: 248}, "INVALID_ARG"), ({2: 258}, "ALIGNMENT"),
        ({16: 0}, "INVALID_ARG"), ({3: -1}, "INVALID_ARG"), ({4: 0}, "INVALID_ARG"), ({4: 3}, "INVALID_ARG"),
        ({4: 4098, 2: 4098 * 64, 16: 4098 * 64}, "UNSUPPORTED"), ({8: -1}, "INVALID_ARG"), ({9: -1}, "INVALID_ARG"),
        ({10: -1}, "INVALID_ARG"), ({11: -1}, "INVALID_ARG"), ({11: 2 ** 30 + 1}, "UNSUPPORTED"),
        ({10: 2 ** 29}, "UNSUPPORTED"), ({8: 2 ** 30}, "UNSUPPORTED"), ({12: P, 13: 0}, "INVALID_ARG"), ({14: 0.0}, "INVALID_ARG"),
        ({14: -1.0}, "INVALID_ARG"), ({14: float("nan")}, "INVALID_ARG"), ({14: float("inf")}, "INVALID_ARG"),
        ({17: None}, "WORKSPACE"), ({18: need - 1}, "WORKSPACE"), ({17: P + 8}, "ALIGNMENT"), ({1: P + 8}, "ALIGNMENT"),
        ({5: P + 2}, "ALIGNMENT"), ({6: P + 1}, "ALIGNMENT"), ({7: P + 2}, "ALIGNMENT"), ({12: P + 2, 13: 1}, "ALIGNMENT")])
    for at in (3, 8, 10):  # no tokens, no sequences
        args = list(good)
        args[at] = 0
        args[1] = args[5] = args[6] = args[7] = args[15] = args[17] = None
        args[18] = 0
        assert f(*args) == L.QE_OK
        assert lib.qe_attention_workspace_bytes(ref(c), 4, *[0 if at == i else v for i, v in ((3, 8), (8, 2), (10, 4))], 4096) == 0


def test_attention_workspace_holds_the_pieces(L):
    """Partials of every row and piece; more tokens never need less."""
    for hd in (64, 128):
        c = _cache(L, head_dim=hd, n_pages=1 << 20)
        last = 0
        for T in (1, 2, 17, 64):
            b = L.qe_attention_workspace_bytes(c, 16, T, 1, T, 1 << 20)
            assert b >= T * 16 * (hd + 2) * 4 and b >= last
            last = 0 if T == 2 else b  # (the form changes with the rows)
    assert L.qe_attention_workspace_bytes(_cache(L, head_dim=80), 4, 8, 2, 4, 4096) == 0


def test_verify_refusals(L):
    lib = L.raw_library()
    f = lib.qe_verify_drafts
    need = lib.qe_verify_workspace_bytes(2, 1000)
    assert need > 0
    # p p_stride draft d_stride vocab row_start n_rows token parent u n_seq max_rows taken path next ws bytes stream
    good = [P, 1000, P, 1000, 1000, P, 8, P, None, P, 2, 4, P, P, P, P, need, None]
    _refused(L, f, good, [
        ({0: None}, "INVALID_ARG"), ({1: 999}, "INVALID_ARG"), ({3: 999}, "INVALID_ARG"), ({4: 0}, "INVALID_ARG"),
        ({4: 2 ** 22 + 1, 1: 2 ** 23, 3: 2 ** 23}, "UNSUPPORTED"), ({5: None}, "INVALID_ARG"), ({6: -1}, "INVALID_ARG"),
        ({7: None}, "INVALID_ARG"), ({8: P}, "UNSUPPORTED"), ({9: None}, "INVALID_ARG"), ({10: -1}, "INVALID_ARG"), ({10: 2 ** 30}, "UNSUPPORTED"),
        ({11: -1}, "INVALID_ARG"), ({11: 1025}, "UNSUPPORTED"), ({12: None}, "INVALID_ARG"), ({13: None}, "INVALID_ARG"),
        ({14: None}, "INVALID_ARG"), ({15: None}, "WORKSPACE"), ({16: need - 1}, "WORKSPACE"), ({0: P + 2}, "ALIGNMENT"),
        ({2: P + 2}, "ALIGNMENT"), ({7: P + 1}, "ALIGNMENT"), ({15: P + 8}, "ALIGNMENT")])
    args = list(good)
    args[10] = 0
    args[5] = args[12] = args[14] = args[15] = None
    assert f(*args) == L.QE_OK
    assert lib.qe_verify_workspace_bytes(1, 0) == 0 and lib.qe_verify_workspace_bytes(2 ** 31 - 1, 2 ** 22) == 0


@pytest.mark.parametrize("kind", ["plain", "linear", "ntk", "yarn"])
@pytest.mark.parametrize("rot,base", [(16, 1e4), (64, 1e4), (128, 1e6), (256, 5e5)])
def test_frequencies(L, kind, rot, base):
    """A power, a quotient and a few products in float64: within 1e-13 relative."""
    at = dict(plain=0, linear=1, ntk=2, yarn=3)[kind]
    f, s = L.qe_rope_freqs(rot, base, at, 4.0, 32768, 1.0, 32.0)
    want, scale = C.freqs(rot, base, kind, 4.0, 32768, 1.0, 32.0)
    assert f.shape == (rot // 2,)
    assert np.allclose(f, want, rtol=1e-13, atol=0)
    assert abs(s - scale) <= 1e-15 * scale
    assert np.all(np.diff(f) < 0) and f[0] <= 1.0
    if kind == "yarn":  # fast pairs keep their speed, slow ones are divided
        plain, _ = C.freqs(rot, base)
        assert f[0] == plain[0]
        assert f[-1] >= plain[-1] / 4 * (1 - 1e-13)


def test_frequency_refusals(L):
    for a in [(0, 1e4), (-16, 1e4), (64, 1.0), (64, float("nan")), (64, float("inf")), (64, 1e4, 4), (64, 1e4, -1),
              (64, 1e4, 1, 0.5), (64, 1e4, 1, float("inf")), (64, 1e4, 3, 4.0, 0.0), (64, 1e4, 3, 4.0, 100.0, 2.0, 2.0),
              (64, 1e4, 3, 4.0, 100.0, float("nan"), 2.0)]:
        with pytest.raises(L.QEError) as e:
            L.qe_rope_freqs(*a)
        assert e.value.status == L.QE_ERR_INVALID_ARG, a
    for rot in (24, 272):
        with pytest.raises(L.QEError) as e:
            L.qe_rope_freqs(rot, 1e4)
        assert e.value.status == L.QE_ERR_UNSUPPORTED
    lib = L.raw_library()
    f = np.zeros(32)
    assert lib.qe_rope_freqs(64, 1e4, 0, 1.0, 0.0, 0.0, 0.0, None, f.ctypes.data) == L.QE_ERR_INVALID_ARG
    assert lib.qe_rope_freqs(64, 1e4, 0, 1.0, 0.0, 0.0, 0.0, f.ctypes.data, None) == L.QE_ERR_INVALID_ARG


def test_bindings_refuse_before_the_library_is_called(L):
    bf = torch.bfloat16
    with pytest.raises(TypeError, match="float64"):
        L.make_rope(torch.zeros(8))
    with pytest.raises(ValueError, match="three"):
        L.make_rope(torch.zeros(8, dtype=torch.float64), sections=(4, 4))
    rope = L.make_rope(torch.zeros(8, dtype=torch.float64))
    assert rope.rot_dim == 16 and rope.n_pos == 1
    x, pos = torch.zeros(3, 2, 64, dtype=bf), torch.zeros(3, dtype=torch.int32)
    with pytest.raises(ValueError, match="device tensors"):
        L.qe_rope_apply(rope, pos, x, x)
    with pytest.raises(TypeError, match="pos must be"):
        L.qe_rope_apply(rope, pos.long(), x, x)
    with pytest.raises(ValueError, match="y must have shape"):
        L.qe_rope_apply(rope, pos, x, x[:2])
    with pytest.raises(ValueError, match="dense within a token"):
        L.qe_rope_apply(rope, pos, x, x.transpose(0, 1).contiguous().transpose(0, 1))
    k = torch.zeros(4, 2, 16, 64, dtype=bf)
    with pytest.raises(TypeError, match="bf16 or int8"):
        L.make_cache(k.float(), k.float())
    with pytest.raises(ValueError, match="scales"):
        L.make_cache(k.to(torch.int8), k.to(torch.int8))
    with pytest.raises(ValueError, match="scales"):
        L.make_cache(k, k, torch.zeros(4, 2, 16), torch.zeros(4, 2, 16))
    with pytest.raises(ValueError, match="v must have shape"):
        L.make_cache(k, k[:2])
    cache = L.make_cache(k, k.clone())
    slot = torch.zeros(3, dtype=torch.int32)
    with pytest.raises(ValueError, match="device tensors"):
        L.qe_kv_append(cache, x, x, slot)
    with pytest.raises(TypeError, match="one type"):
        L.qe_kv_append(cache, x, x.float(), slot)
    with pytest.raises(ValueError, match="come together"):
        L.qe_kv_append(cache, x, x, slot, q=x)
    with pytest.raises(ValueError, match="k must have shape"):
        L.qe_kv_append(cache, x[:, :1], x, slot)
    i = torch.zeros(2, dtype=torch.int32)
    pages = torch.zeros(1, 4, dtype=torch.int32)
    with pytest.raises(ValueError, match="device tensors"):
        L.qe_attention(cache, x, i, i[:1], pages, 3, 64, x.clone(), None)
    with pytest.raises(TypeError, match="must be bf16"):
        L.qe_attention(cache, x.float(), i, i[:1], pages, 3, 64, x.clone(), None)
    with pytest.raises(ValueError, match="pages must have shape"):
        L.qe_attention(cache, x, i, i[:1], pages[0], 3, 64, x.clone(), None)
    with pytest.raises(ValueError, match="heads of"):
        L.qe_attention(cache, x[..., :32], i, i[:1], pages, 3, 64, x.clone(), None)
    p = torch.zeros(2, 10)
    with pytest.raises(TypeError, match="float32"):
        L.qe_verify_drafts(p.to(bf), i, i, p[:, 0].contiguous(), i[:1], i, i[:1], i)
    with pytest.raises(ValueError, match="token must have shape"):
        L.qe_verify_drafts(p, i, i[:1], p[:, 0].contiguous(), i[:1], i, i[:1], i)


def test_oracle_rotation_keeps_lengths_and_shifts():
    """A rotation keeps a pair's length, and products of queries and keys depend on their distance alone."""
    rng = np.random.default_rng(3)
    f, _ = C.freqs(32, 1e4)
    q, k = rng.standard_normal((2, 5, 1, 48))
    pos = rng.integers(0, 1000, (1, 5))
    for pairs in (False, True):
        a, b = C.rope(q, pos, f, pairs), C.rope(k, pos + 7, f, pairs)
        assert np.allclose(np.linalg.norm(a, axis=-1), np.linalg.norm(q, axis=-1))
        assert np.array_equal(a[..., 32:], q[..., 32:])
        a2, b2 = C.rope(q, pos + 100, f, pairs), C.rope(k, pos + 107, f, pairs)
        assert np.allclose((a * b).sum(-1), (a2 * b2).sum(-1))
    # pair 0 turns by one radian per position
    one = np.zeros((1, 1, 32))
    one[..., 0] = 1.0
    y = C.rope(one, np.array([[2]]), f)
    assert np.allclose(y[0, 0, [0, 16]], [np.cos(2), np.sin(2)])


def test_oracle_verification_by_hand():
    p = np.array([[0.5, 0.3, 0.2], [0.1, 0.2, 0.7], [0.6, 0.4, 0.0]], np.float32)
    tok = np.array([9, 0, 2])
    # both drafts chosen: accepted when u < p; u0 then draws from the last row
    assert C.verify(p, tok, np.array([0.59, 0.49, 0.69])) == ([1, 2], 0)
    assert C.verify(p, tok, np.array([0.61, 0.49, 0.69])) == ([1, 2], 1)
    assert C.verify(p, tok, np.array([0.59, 0.51, 0.0])) == ([], 1)  # token 0 refused: 0.3 and 0.2 left
    assert C.verify(p, tok, np.array([0.61, 0.51, 0.0])) == ([], 2)
    # two siblings at the root: the second's probability is taken of what the first left
    par = np.array([-1, 0, 0])
    assert C.verify(p, np.array([9, 0, 1]), np.array([0.0, 0.9, 0.59]), parent=par) == ([2], 0)
    assert C.verify(p, np.array([9, 0, 1]), np.array([0.0, 0.9, 0.61]), parent=par) == ([], 2)
    # a chain with distributions: token 0 drawn with 0.8 against 0.5, refused: drawn from (0, 0.2, 0.1)
    d = np.array([[0, 0, 0], [0.8, 0.1, 0.1], [0.1, 0.1, 0.8]], np.float32)
    assert C.verify(p, tok, np.array([0.66, 0.63, 0.0]), draft_p=d) == ([], 1)
    assert C.verify(p, tok, np.array([0.67, 0.63, 0.0]), draft_p=d) == ([], 2)
    assert C.verify(p, tok, np.array([0.0, 0.62, 0.88]), draft_p=d) == ([1], 1)  # then from (0, 0.1, 0)
    assert C.verify(p, tok, np.array([0.0, 0.62, 0.87]), draft_p=d) == ([1, 2], 0)


def test_oracle_verification_keeps_the_distribution():
    """Whatever the drafts, the first token comes out with the target's probabilities."""
    rng = np.random.default_rng(0)
    p = np.array([[0.5, 0.2, 0.2, 0.1]] * 3, np.float32)
    d = np.array([[0, 0, 0, 0], [0.1, 0.6, 0.1, 0.2], [0.25] * 4], np.float32)
    n, count = 20000, np.zeros((2, 4))
    for _ in range(n):
        u = rng.random(3)
        x = rng.choice(4, p=d[1].astype(np.float64) / d[1].astype(np.float64).sum())
        path, nxt = C.verify(p[:2], np.array([0, x]), u[:2], draft_p=d[:2])
        count[0, x if path else nxt] += 1
        path, nxt = C.verify(p, np.array([0, 1, 0]), u, parent=np.array([-1, 0, 0]))
        count[1, (1, 0)[path[0] - 1] if path else nxt] += 1
    # five standard deviations of a share of 20000 draws: 5 / (2 sqrt(20000)) = 0.018
    assert np.all(np.abs(count / n - p[0]) < 0.018)
