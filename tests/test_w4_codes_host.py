"""The arithmetic behind the 4-bit codes, over every case it depends on: a reciprocal that is a few units off and two
roundings give the codes of the exact quotient (no GPU; fp32 is rounded from float64, exactly)."""

import numpy as np
import torch

from oracle import few_bits_oracle as F

ULPS = range(-3, 4)  # the reciprocal's error: the approximate one is documented within 2 units in the last place


def f32(v):
    return np.asarray(v, np.float64).astype(np.float32).astype(np.float64)


def reciprocals(s):
    """1 / s rounded to fp32, and its neighbours."""
    r = f32(1.0 / s)
    return [r + k * np.ldexp(1.0, np.frexp(r)[1] - 24) for k in ULPS]


def rounded(x, r):
    """round(x r) by way of 3 * 2^10, whose unit in the last place in fp32 is 2^-12, and then an integer."""
    c = f32(x * r + 3072.0) - 3072.0  # one fused multiply-add; x r has 32 bits and the sum 44, exact in float64
    return f32(c + 12582920.0) - 12582920.0


def test_a_quotient_is_a_tie_or_well_away_from_one():
    """Significands a and b of 8 bits: the distance of a 2^e / b <= 7.5 from every k + 1/2 is 0 or at least 2^-10."""
    a, b = np.arange(128, 256)[:, None], np.arange(128, 256)[None, :]
    for e in range(-12, 4):
        q2 = (a * 2.0 ** (e + 1)) / b  # twice the quotient: distance from odd integers
        odd = 2 * np.floor(q2 / 2) + 1
        exact = np.abs(a * 2.0 ** (e + 1) - odd * b) / (2 * b)  # the numerator is exact
        keep = q2 <= 15
        assert ((exact == 0) | (exact >= 2.0 ** -10))[keep].all()


def test_codes_over_every_significand():
    """Scales of full precision: every pair of significands and every exponent of a quotient up to 7.5."""
    a, b = np.arange(128, 256, dtype=np.float64)[:, None], np.arange(128, 256, dtype=np.float64)[None, :]
    for r in reciprocals(b):
        for e in range(-12, 4):
            x = a * 2.0 ** e
            keep = x <= 7.5 * b
            assert np.array_equal(rounded(x, r)[keep], np.rint(x / b)[keep]), e


def test_codes_of_scales_with_few_bits():
    """Scales below bf16's normal range are multiples b of 2^-133 and so are the weights: quotients up to 10, clamped
    where rounding made the scale that much smaller than max / 7."""
    for b in range(1, 128):
        w = np.arange(0, 11 * b + 1, dtype=np.float64)
        w = w[w <= 10 * b + 3]
        for r in reciprocals(np.float64(b)):
            assert np.array_equal(np.clip(rounded(w, r), -8, 7), np.clip(np.rint(w / b), -8, 7)), b


def test_the_scale_over_every_significand():
    """max / 7 is never so near a tie between bf16 neighbours that the product with fp32's 1 / 7 rounds otherwise, in the
    normal range and below it."""
    seventh = f32(1.0 / 7.0)
    for a, e in [(np.arange(128, 256), 0), (np.arange(128, 256), -60), (np.arange(0, 256), -133)]:
        m = a * 2.0 ** e
        product = (torch.tensor(m, dtype=torch.float32) * float(seventh)).double().numpy()
        assert np.array_equal(F.bf16_round(product), F.bf16_round(m / 7.0))


def test_bf16_round_below_the_normal_range():
    rng = np.random.default_rng(5)
    v = np.concatenate([rng.normal(size=4096) * 2.0 ** rng.integers(-136, -120, 4096),
                        np.arange(-9, 10) * 2.0 ** -134])
    v = v.astype(np.float32).astype(np.float64)
    ref = torch.tensor(v, dtype=torch.float32).to(torch.bfloat16).double().numpy()
    assert np.array_equal(F.bf16_round(v), ref)


def test_the_tests_see_a_code_that_is_off():
    """A reciprocal of 11 bits does change codes: the tests above are not passed by anything."""
    a, b = np.arange(128, 256, dtype=np.float64)[:, None], np.arange(128, 256, dtype=np.float64)[None, :]
    r = (1.0 / b).astype(np.float16).astype(np.float64)
    x = a * 4.0
    keep = x <= 7.5 * b
    assert not np.array_equal(rounded(x, r)[keep], np.rint(x / b)[keep])
