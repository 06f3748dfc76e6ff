"""Calls of the cache and attention bindings that their C arguments cannot carry (no GPU needed)."""

import pytest
import torch


@pytest.fixture(scope="module")
def L():
    from quantized_linear_moe_amd import _libqe
    return _libqe


def _attention(L, **kw):
    k = torch.zeros(4, 2, 16, 64, dtype=torch.bfloat16)
    x, i = torch.zeros(3, 2, 64, dtype=torch.bfloat16), torch.zeros(2, dtype=torch.int32)
    a = dict(max_q=3, max_kv=64)
    a.update(kw)
    L.qe_attention(L.make_cache(k, k.clone()), x, i, i[:1], torch.zeros(1, 4, dtype=torch.int32), out=x.clone(), ws=None, **a)


def test_tree_without_words(L):
    """An empty tree's address is NULL, which the library takes for no tree."""
    with pytest.raises(ValueError, match="tree has no words"):
        _attention(L, tree=torch.zeros(3, 0, dtype=torch.int32))
    with pytest.raises(ValueError, match="device tensors"):
        _attention(L, tree=torch.zeros(3, 1, dtype=torch.int32))


@pytest.mark.parametrize("n", [2 ** 31, 2 ** 32, 2 ** 32 + 64])
def test_bounds_past_32_bits(L, n):
    """ctypes would pass the low 32 bits on: 2^32 keys at most would leave out all of them."""
    for name in ("max_q", "max_kv"):
        with pytest.raises(ValueError, match=name):
            _attention(L, **{name: n})
    k = torch.zeros(4, 2, 16, 64, dtype=torch.bfloat16)
    cache = L.make_cache(k, k.clone())
    assert L.qe_attention_workspace_bytes(cache, 4, 8, 2, 4, n + 4096) == 0
    p, i = torch.zeros(2, 10), torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError, match="max_rows"):
        L.qe_verify_drafts(p, i, i, p[:, 0].contiguous(), i[:1], i, i[:1], i, max_rows=n)
