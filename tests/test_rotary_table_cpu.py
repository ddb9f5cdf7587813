"""The rotary table against the error that the header states for it, with the
frequencies worked out in 60 decimal digits."""
import random
from decimal import Decimal as Dec
from decimal import localcontext

import pytest

TWO_PI = 2 * Dec("3.14159265358979323846264338327950288419716939937510582097494459230781640628620899")


@pytest.fixture(scope="module")
def S():
    from serving_sd_verify_gb300 import build, sd_verify
    build.build()
    sd_verify.load()
    return sd_verify


def turns_per_position(i, R, theta, scaling, factor, original, low, high):
    theta, f = Dec(theta), Dec(factor)
    if scaling == "ntk":
        theta *= (Dec(R) / Dec(R - 2) * f.ln()).exp()
    w = (Dec(-2 * i) / Dec(R) * theta.ln()).exp()
    if scaling == "linear":
        w /= f
    if scaling in ("parts", "yarn"):
        g = min(Dec(1), max(Dec(0), (original * w / TWO_PI - Dec(low)) / (Dec(high) - Dec(low))))
        w = (1 - g) * w / f + g * w
    return w / TWO_PI


@pytest.mark.parametrize("scaling", ["none", "linear", "ntk", "parts", "yarn"])
def test_words_are_as_good_as_the_header_says(S, scaling):
    """A word is the fraction of w / (2 pi) cut off at 2^-64, w right to e = 2^-49: the exponent's rounding
    times ln theta (23 where theta, stretched, is below 10^10), the power and the two divisions are 16
    halves of an ulp.  Where frequencies are blended, a relative error d of the turns over the original
    context moves the result by up to d (1 + factor low / (high - low))."""
    rng = random.Random(scaling)
    for _ in range(60):
        R, theta = 2 * rng.randint(2, 128), rng.choice([1e4, 5e5, 1e6, 1e7, 1e-3, rng.uniform(2, 1e8)])
        factor, low, high = rng.choice([1.0, 2.0, 4.0, 8.0, rng.uniform(1, 64)]), 1.0, rng.choice([4.0, 32.0])
        original = rng.choice([4096, 8192, 32768])
        words, _ = S.sd_rotary_table(R, theta, scaling=scaling, factor=factor, original_max=original, low=low, high=high)
        e = 2.0 ** -49 * (2 + factor * low / (high - low) if scaling in ("parts", "yarn") else 1)
        with localcontext() as c:
            c.prec = 60
            for i, word in enumerate(words.tolist()):
                t = turns_per_position(i, R, theta, scaling, factor, original, low, high)
                d = abs(Dec(word % 2 ** 64) / Dec(2 ** 64) - t % 1)
                d = float(min(d, 1 - d))
                assert d <= e * float(t) + 2.0 ** -64, (R, theta, factor, i, d / (float(t) * 2.0 ** -53))
