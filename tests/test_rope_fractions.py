"""Rotary frequencies against decimals of 60 digits: a position of 31 bits multiplies
the fraction's error, so its 64 bits all count."""

import decimal

import pytest

import autoregressive_speech_token_gb300 as pkg

TWO_PI = decimal.Decimal("6.28318530717958647692528676655900576839433879875021164194989")


@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("theta", [1e4, 1e6, 5e5, 10000.1, 1.0000001, 1.5, 2.0, 1e15, 1e300])
def test_fractions_have_64_bits(hd, theta):
    """Every fraction within one unit of 2^-64 of a turn: rounded down, with an error of the sum of two doubles below
    2^-95 of it."""
    from autoregressive_speech_token_gb300 import build
    build.build()
    rope = pkg.sd_rope_init(hd, theta)
    with decimal.localcontext() as c:
        c.prec = 60
        ln = decimal.Decimal(theta).ln()
        for i in range(hd // 2):
            want = (-2 * i * ln / hd).exp() / TWO_PI * 2 ** 64
            assert -1 <= rope.turn[i] - want <= decimal.Decimal("0.001"), (i, rope.turn[i], want)
