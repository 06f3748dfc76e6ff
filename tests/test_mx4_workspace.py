"""The plan that a microscaled product's shape selects, read from its workspace (no GPU needed).

A linear without corrections has in its workspace the codes and scales of its tokens, three vectors of one int32 per
token (scores, routes, order), two small tables, the float32 partials of a split sum, and, for tiles of 128 tokens
and more, the activations' tiles: rows rounded up to 32, 17/32 bytes per element.
"""

import pytest


@pytest.fixture(scope="module")
def L():
    from quantized_linear_moe_amd import _libqe
    return _libqe


def _align(n):
    return (n + 255) // 256 * 256


@pytest.mark.parametrize("T,d_in,d_out,tiles,splits", [
    (70, 29568, 6160, True, 4), (128, 29568, 8192, True, 4), (129, 29568, 8192, True, 2), (65, 16384, 24592, True, 1),
    (100, 8320, 24592, True, 1), (200, 1024, 32784, True, 1), (256, 1024, 32784, True, 1), (257, 1024, 32784, True, 1),
    (180, 8320, 32784, True, 1), (64, 29568, 8192, False, 4), (12, 29568, 8192, False, 1), (250, 8320, 64, False, 8),
])
def test_plan(L, T, d_in, d_out, tiles, splits):
    lin = L.make_linear(d_in, d_out, 4, 4, 0, 0, 0)
    rows = (T + 31) // 32 * 32
    want = _align(T * d_in // 2) + _align(T * d_in // 32) + 3 * _align(4 * T) + 2 * _align(128)
    want += _align(4 * splits * T * d_out) if splits > 1 else 0
    want += _align(rows * d_in // 2) + _align(rows * d_in // 32) if tiles else 0
    assert L.qe_workspace_bytes(lin, T) == want
