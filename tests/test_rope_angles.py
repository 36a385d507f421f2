"""How far the angle of the position rotation is off, as include/pkv.h has it: the kernel's integer
arithmetic (position times a 64-bit fraction of a turn, its top 32 bits as fp32) against exact
fractions, on the CPU."""
import random
import struct
from fractions import Fraction

import numpy as np
import pytest

import paged_kv_attention_22_gb300 as pkv
from paged_kv_attention_22_gb300 import build as pkv_build

PI = Fraction(31415926535897932384626433832795028841971693993751, 10 ** 49)


@pytest.fixture(scope="module")
def L():
    pkv_build.build()
    return pkv.lib()


def _off(position, turns, frequency):
    """Turns between the angle that sincospi gets and position * frequency."""
    top = (position * turns % 2 ** 64) >> 32
    halves = np.float32(np.int64(top - (top >> 31 << 32)).astype(np.int32)) * np.float32(2.0 ** -31)
    off = Fraction(float(halves)) / 2 - position * Fraction(frequency) / (2 * PI)
    return abs(off - round(off))


def test_angles_are_as_near_as_the_header_says(L):
    rng = random.Random(1)
    near = 0
    for _ in range(20):
        f = [1.0] + [10.0 ** -rng.uniform(0, 6) * rng.choice([1, -1]) for _ in range(63)]
        turns = struct.unpack("<iifi64Q", pkv.rope(128, frequencies=f).data)[4:]
        for w, x in zip(turns, f):
            for position in (rng.randrange(1 << 17), -rng.randrange(1 << 24), rng.randrange(1 << 31), (1 << 31) - 1, -(1 << 31)):
                # 24 bits of half a turn either way, half a step of them, 2^-26 of a turn; the top 32
                # bits, 2^-32; and 2 pi's, the division's and the fraction's roundings, by position
                off = _off(position, w, x)
                bound = Fraction(1, 2 ** 26) + Fraction(1, 2 ** 32) + abs(position) * (abs(Fraction(x)) / 2 ** 54 + Fraction(1, 2 ** 64))
                assert off <= bound, (position, x, float(off), float(bound))
                near = max(near, off / Fraction(1, 2 ** 32) if abs(position) < 1 << 17 else 0)
    assert near > 8  # it is not 2^-32
