"""Host-only: the binding's fractions of a turn against whole-number arithmetic on pi."""
import random
from fractions import Fraction

import pytest

from hybrid_ssm_gated_gb300 import kv
from tests.turns_ref import fraction, slack


@pytest.mark.parametrize("base", [1e4, 1e6, 5e5])
@pytest.mark.parametrize("half", [16, 32, 64, 128])
def test_fractions_of_a_turn(base, half):
    freq = [base ** (-i / half) for i in range(half)] + [random.Random(half).uniform(-9, 9) for _ in range(50)]
    turns = kv.Rotary(freq, device="cpu").turns.tolist()
    for f, t in zip(freq, turns):
        off = (t - fraction(f) * 2 ** 64) % 2 ** 64  # both ways round
        assert min(off, 2 ** 64 - off) <= slack(f) * 2 ** 64


def test_the_reference():
    assert abs(fraction(1.0) - Fraction(15915494309189533577, 10 ** 20)) < Fraction(1, 10 ** 19)  # 1 / (2 pi)
    assert slack(1.0) < Fraction(1, 2 ** 55)
