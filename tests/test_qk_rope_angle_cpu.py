"""The angle of the rotation, step by step in whole numbers, against the bounds that the header and the kernel state.

A frequency f = m 2^-s (m below 2^24) as turns per position is floor(m c 2^-s) of 2^64 to a turn, c = floor(2^64 / 2 pi). 2^64 /
2 pi ends in .4962, so for f up to 1 the number is short by less than .4963 f + 1 < 1.4963 units, and times a position
of up to 2^31 by less than 1.4963 2^-33 < 2^-32.4 of a turn. Its top 32 bits, rounded, are off by another 2^-33 at most: 2^-31.6
together. As a float with 24 bits the largest of them (from 2^30 on) are rounded by up to 2^6 of 2^32 to a turn: 2^-26, and
2^-25.9 in all."""
import os
import random
import struct
from fractions import Fraction

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
PI = Fraction(314159265358979323846264338327950288419716939937510582097494459230781640628620899, 10 ** 80)
TURN = (1 << 64)
C = int(TURN / (2 * PI))


def _f32(x):
    return struct.unpack("f", struct.pack("f", x))[0]


def _parts(f):
    """f = ± m 2^-s."""
    bits = struct.unpack("I", struct.pack("f", f))[0]
    field = bits >> 23 & 255
    return (bits & 0x7FFFFF) | (0x800000 if field else 0), 150 - max(field, 1), bits >> 31


def _turns(f):
    m, s, negative = _parts(f)
    t = (m * C << -s if s <= 0 else m * C >> s) % TURN
    return -t % TURN if negative else t


def _off(a, b):
    """Distance of two angles in turns."""
    d = (a - b) % 1
    return min(d, 1 - d)


def test_the_constant_is_that_of_the_source():
    source = open(os.path.join(ROOT, "dense_bf16_gemm_02_gb300", "csrc", "qk_rope.cuh")).read()
    assert f"0x{C:X}ull" in source
    assert Fraction(4962, 10000) < TURN / (2 * PI) - C < Fraction(4963, 10000)


def test_the_bounds_of_the_angle():
    rng = random.Random(5)
    freqs = [1.0, -1.0, _f32(1 - 2.0 ** -24), 2.0 ** -126, 2.0 ** -149, 0.5] + [_f32(rng.uniform(0.5, 1)) for _ in range(40)]
    freqs += [_f32(10000.0 ** -rng.random()) * rng.choice((1, -1)) for _ in range(40)] + [_f32(2.0 ** rng.uniform(-60, 0)) for _ in range(40)]
    places = [0, 1, -1, 2 ** 31 - 1, -2 ** 31, 1 - 2 ** 31, 10 ** 6] + [rng.randrange(-2 ** 31, 2 ** 31) for _ in range(60)]
    places += [2 ** 31 - 1 - rng.randrange(1000) for _ in range(20)]
    worst = [Fraction(0)] * 3
    for f in freqs:
        m, s, negative = _parts(f)
        per = Fraction(-m if negative else m) / (Fraction(2) ** s) / (2 * PI)
        assert abs(Fraction(m, 1) / Fraction(2) ** s) == abs(Fraction(f))
        for at in places:
            turn = _turns(f) * at % TURN
            top = (turn + (1 << 31) >> 32) % (1 << 32)
            top -= (1 << 32) if top >= 1 << 31 else 0
            used = Fraction(_f32(float(top)))
            for i, got in enumerate((Fraction(turn, TURN), Fraction(top, 1 << 32), used / (1 << 32))):
                worst[i] = max(worst[i], _off(got, per * at))
    bounds = 2.0 ** -32.4, 2.0 ** -31.6, 2.0 ** -25.9
    assert all(float(w) < b for w, b in zip(worst, bounds)), [float(w) for w in worst]
    assert float(worst[2]) > 2.0 ** -26.5               # (the rounding to 24 bits is what it comes to)
