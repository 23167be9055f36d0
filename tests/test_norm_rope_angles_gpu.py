"""Angles of far positions against an exact reduction.

Pairs (1, 0) without a norm come out as (cos, sin).  An angle is held to 2^-28 of a turn
(the float of what is left of the nearest quarter turn), 2^-32 (the product's leading 32
bits) and 2^-33 (a unit of 2^-64 times a position of 2^31): under 7 * 2^-28 radians together.
Cosine and sine are good to 2 ulp of FP32, and are rounded once to BF16, half a step 2^-8.
Positions are searched whose angles lie near
quarter turns, where BF16 has steps fine enough to show an angle that is off."""
import math
from fractions import Fraction

import numpy as np
import pytest
import torch

from tests.gpu_common import built_library

FREQS = [1.0, 40.0, -9.0, 0.7, 1e-3, 3.1e4, 2.0 ** 40, 7.0, -3e38, 1.7e25, 1e-6, 1e-40]


def per_turn(bits=400):
    """1 / 2 pi, by Machin's formula."""
    def atan_of_inverse(x):
        term = total = (1 << bits) // x
        n, sign = 3, -1
        while term:
            term //= x * x
            total += sign * (term // n)
            n, sign = n + 2, -sign
        return total
    return Fraction(1 << bits, 8 * (4 * atan_of_inverse(5) - atan_of_inverse(239)))


PER_TURN = per_turn()


def exact(pos, freq):
    """cos and sin of pos * freq."""
    turns = Fraction(pos) * Fraction(freq) * PER_TURN
    quarter = math.floor(turns * 4 + Fraction(1, 2))
    a = float(turns - Fraction(quarter, 4)) * 2.0 * math.pi
    return [(math.cos(a), math.sin(a)), (-math.sin(a), math.cos(a)), (-math.cos(a), -math.sin(a)),
            (math.sin(a), -math.cos(a))][quarter % 4]


def telling_positions():
    """Of each frequency and span of positions, those whose angles lie nearest a quarter turn."""
    out = [0, 1, -1, 2 ** 31 - 1, -2 ** 31]
    for f in FREQS:
        turn = int(Fraction(float(np.float32(f))) * PER_TURN % 1 * 2 ** 64)
        for first in (2 ** 31 - 2 ** 18, -2 ** 31, 10 ** 8, 10 ** 7, -10 ** 6):
            pos = np.arange(first, first + 2 ** 18, dtype=np.int64)
            with np.errstate(over="ignore"):
                left = (pos.astype(np.uint64) * np.uint64(turn)) << np.uint64(2)
            near = np.abs(left.astype(np.int64).astype(np.float64))
            out += [int(x) for x in pos[np.argsort(near)[:4]]]
    return out


def test_the_reduction_of_the_test():
    """Against the library's own cosine and sine, where these are good enough."""
    c, s = exact(710, 1.0)
    assert abs(s - math.sin(710.0)) < 1e-12 and abs(c - math.cos(710.0)) < 1e-12
    c, s = exact(1000003, 0.5)
    assert abs(s - math.sin(500001.5)) < 1e-9 and abs(c - math.cos(500001.5)) < 1e-9


@pytest.mark.gpu
@pytest.mark.parametrize("F", [16, 12])                    # sixteen elements a lane, and eight
@pytest.mark.parametrize("interleaved", [False, True])
def test_far_positions_to_the_bound(F, interleaved):
    fw = built_library()
    freqs = (FREQS + [0.25, -0.125, 3.0, 100.0])[:F]
    pos = telling_positions()
    x = torch.zeros(len(pos), 1, 64, dtype=torch.bfloat16, device="cuda")
    a = [2 * i if interleaved else i for i in range(F)]
    b = [2 * i + 1 if interleaved else i + F for i in range(F)]
    x[:, :, a] = 1.0
    q, k = fw.qk_norm_rope(x, x, torch.tensor(pos, dtype=torch.int32, device="cuda"),
                           torch.tensor(freqs, device="cuda"), interleaved=interleaved)
    assert fw.device_status() == 0 and torch.equal(q, k)
    got = q[:, 0].double().cpu().numpy()
    worst = 0.0
    for i, f in enumerate(np.float32(freqs)):
        want = np.array([exact(p, float(f)) for p in pos])
        err = np.abs(np.stack([got[:, a[i]], got[:, b[i]]], -1) - want)
        bound = (2.0 ** -8 + 2.0 ** -21) * np.abs(want) + 7.0 * 2.0 ** -28
        worst = max(worst, (err / bound).max())
    assert worst <= 1.0, worst
