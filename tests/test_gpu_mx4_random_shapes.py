"""The forward of microscaled linears over seeded random shapes: 1 to 700 tokens, 128 to 32768 input channels, outputs
of 16 to 40000, every kind of rank and expert count, both input types, and widths past 32768 (which only a_bits 4 and
16 take).  The checks and tolerances are those of test_gpu_mx4_forward.py.
"""

import math
import random

import pytest
import torch

import test_gpu_mx4_forward as forward

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


def _shapes(count, seed):
    r = random.Random(seed)
    log = lambda lo, hi: min(hi, max(lo, round(math.exp(r.uniform(math.log(lo), math.log(hi))))))  # noqa: E731
    out = []
    while len(out) < count:
        d_in, d_out = 128 * log(1, 256), 16 * log(1, 2500)
        if d_in * d_out > 2 ** 27:
            continue
        n_r = r.choice((0, 1, 2, 4, 8, 13, 16))
        out.append((r.choice((log(1, 64), log(17, 300), log(60, 700))), d_in, d_out, r.choice((0, 1, 16, 32, 33, 64)), n_r,
                    r.choice((1, 8, 32, 48, 64)) if n_r else 0, r.choice((BF, BF, BF, F32))))
    return out


SHAPES = _shapes(40, 6) + [(1, 65664, 64, 32, 8, 32, BF), (16, 65664, 48, 8, 2, 64, F32), (17, 65664, 64, 32, 8, 32, BF),
                           (100, 65664, 1552, 32, 8, 32, BF), (300, 65664, 1040, 0, 16, 64, BF), (3, 262144, 32, 0, 4, 8, BF)]


@pytest.fixture(scope="module")
def Q():
    import quantized_linear_moe_amd as q
    return q


@pytest.mark.parametrize("shape", SHAPES, ids=forward.ids)
def test_codes(Q, shape):
    forward.test_codes(Q, shape)


@pytest.mark.parametrize("shape", [s for s in SHAPES if s[3] or s[4]], ids=forward.ids)
def test_routes_and_corrections(Q, shape):
    forward.test_routes_and_corrections(Q, shape)
