"""How far the table of the rotation's frequencies is off: 2^-52 of a frequency (two roundings of 2^-53, 1 / (2 pi)
and the product with it) and the 2^-64 of a turn that the table ends with."""

from fractions import Fraction

import numpy as np

import sparse_attention_decode_msa_gb300 as msa
from sparse_attention_decode_msa_gb300 import build

PI = Fraction("3.14159265358979323846264338327950288419716939937510582097494459230781640628620899")


def test_a_frequency_is_off_by_two_roundings():
    build.build()
    rng = np.random.default_rng(1)
    radians = np.concatenate([10000.0 ** (-np.arange(64) / 64), rng.uniform(0, 7, 500), 10.0 ** rng.uniform(-12, 9, 500)])
    radians = np.concatenate([radians, -radians])
    got = msa.rope_frequencies(radians.tolist()).numpy().astype(np.uint64)
    for f, t in zip(radians.tolist(), got.tolist()):
        want = Fraction(f) / (2 * PI)
        off = (Fraction(t, 2 ** 64) - want + Fraction(1, 2)) % 1 - Fraction(1, 2)
        assert abs(off) <= abs(want) * Fraction(1, 2 ** 52) + Fraction(1, 2 ** 64), f
