"""The cache's writer divides by 15 as a product with the reciprocal and Markstein's correction
(csrc/kv_append.cu: over15): equal to the rounded quotient for every finite 16-bit value, in
rational arithmetic."""
from fractions import Fraction

import numpy as np
import pytest


def rn32(x):
    """A rational rounded to fp32 (nearest, ties to even; subnormals too), as a rational."""
    if x == 0:
        return x
    n, d = abs(x.numerator), x.denominator
    e = n.bit_length() - d.bit_length()  # floor(log2) or one more
    if (n << max(-e, 0)) < (d << max(e, 0)):
        e -= 1
    unit = max(e - 23, -149)
    n, d = (n << -unit, d) if unit < 0 else (n, d << unit)
    q, r = divmod(n, d)
    q += 2 * r > d or (2 * r == d and q & 1)
    y = Fraction(q) * (Fraction(2) ** unit)
    return y if x > 0 else -y


def values(dtype):
    bits = np.arange(1 << 15, dtype=np.uint32)  # the sign changes nothing: every step is odd
    x = (bits << 16).view(np.float32) if dtype == "bf16" else bits.astype(np.uint16).view(np.float16).astype(np.float32)
    return x[np.isfinite(x)]


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_division_by_fifteen(dtype):
    inv = rn32(Fraction(1, 15))
    x = values(dtype)
    assert len(x) > 31000
    for v in x.tolist():
        f = Fraction(v)
        q = rn32(f * inv)
        r = rn32(f - 15 * q)
        assert rn32(r * inv + q) == rn32(f / 15), v


def test_rounding():
    g = np.random.default_rng(0)
    d = np.concatenate([g.standard_normal(2000) * 2.0 ** g.integers(-140, 120, 2000), [1 + 2.0 ** -24, 1 + 3 * 2.0 ** -24, 2.0 ** -150, 3 * 2.0 ** -150]])
    with np.errstate(under="ignore"):
        for v in d:
            assert float(rn32(Fraction(float(v)))) == float(np.float32(v))
