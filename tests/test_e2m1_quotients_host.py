"""Codes and scales of E2M1 rows at their borders: the oracle's divisions and a
binary32 restatement of the kernels' division-free forms (pkv_device.cuh,
side_of_quotient) against exact decisions (no GPU)."""

import numpy as np
import pytest

from oracle import formats as F

from .e2m1_exact import BORDERS, E4M3, SCALES, around, exact_codes, exact_scale, near_borders

f32 = np.float32


# ------------------------------------------------ the kernels' form in binary32

def kept12(y):
    """Rounded to 12 bits after the point, ties away from zero."""
    return ((y.astype(f32).view(np.uint32) + np.uint32(0x400)) & np.uint32(0xFFFFF800)).view(f32)


def fma(a, b, c):
    """a b + c of binary32 in one rounding.  a b has at most 48 bits; where binary64 does not hold the sum, the
    sum's error (exact, by two-sum) moves a result that lies on a tie of binary32 off it."""
    p, c = a.astype(np.float64) * b.astype(np.float64), c.astype(np.float64)
    s = p + c
    bb = s - p
    err = (p - (s - bb)) + (c - bb)
    s = np.where(err == 0, s, np.where((s.view(np.int64) & 0x1FFFFFFF) == 0x10000000,
                                       np.nextafter(s, np.where(err > 0, np.inf, -np.inf)), s))
    return s.astype(f32)


def side_of_quotient(x, s, r):
    y = kept12((x * r).astype(f32))
    return fma(fma(-y, s, x), r, y)


def reciprocals(s):
    """1 / s in binary32 and its neighbours: the hardware's is off by at most one last place."""
    r = (f32(1.0) / s.astype(f32)).astype(f32)
    for d in (-1, 0, 1):
        yield (r.view(np.int32) + np.int32(d)).view(f32)


# ------------------------------------------------------------------- tests

def test_the_exact_decision_itself():
    x = np.array([0.0, 0.25, 0.2500001, 0.75, 0.7499999, 1.25, 1.75, 2.5, 3.5, 5.0, 5.000001, 1e30, -0.75, -0.0], dtype=f32)
    assert exact_codes(x, 1.0).tolist() == [0, 0, 1, 2, 1, 2, 4, 4, 6, 6, 7, 7, 10, 8]
    a = np.array([0.0, 6 * 2.0 ** -10, 6 * 2.0 ** -9, 9 * 2.0 ** -9, 6.0, 6 * 1.0625, 6 * 1.1875, 2688.0, 1e30, np.inf], dtype=f32)
    assert exact_scale(a).tolist() == [0, 0, 1, 2, 0x38, 0x38, 0x3A, 0x7E, 0x7E, 0x7E]


def test_the_oracle_decides_as_the_exact_quotient():
    x, s = near_borders()
    assert (F.e2m1_encode(F.f32_div(x, s.astype(f32))) == exact_codes(x, s)).all()
    a = around(6.0 * np.unique(np.concatenate([E4M3[1:], (E4M3[1:] + E4M3[:-1]) / 2])), range(-4, 5)).ravel()
    assert (F.e4m3_encode(F.f32_div(a, f32(6.0))) == exact_scale(a)).all()


@pytest.mark.parametrize("off", [1 + 2.0 ** -21, 1 - 2.0 ** -21, 1 + 2.0 ** -23, 1 - 2.0 ** -23])
def test_quotients_a_little_off_are_noticed(off):
    x, s = near_borders()
    y = (x.astype(np.float64) / s * off).astype(f32)
    assert (F.e2m1_encode(y) != exact_codes(x, s)).sum() > 100


def test_sides_of_quotients_of_values_beside_borders():
    x, s = near_borders(range(-40, 41))
    want, s = exact_codes(x, s), s.astype(f32)
    for r in reciprocals(s):
        y = side_of_quotient(x, s, r)
        assert (F.e2m1_encode(y) == want).all()
    a = around(6.0 * np.unique(np.concatenate([E4M3[1:], (E4M3[1:] + E4M3[:-1]) / 2])), range(-40, 41)).ravel()
    r = np.full_like(a, f32(0.16666667))
    assert (F.e4m3_encode(side_of_quotient(a, np.full_like(a, f32(6.0)), r)) == exact_scale(a)).all()


def test_sides_of_quotients_anywhere():
    rng = np.random.default_rng(5)
    s = rng.choice(SCALES, 1_000_000).astype(f32)
    x = (np.exp2(rng.uniform(-12, 3, s.size)) * s).astype(f32) * rng.choice([-1, 1], s.size).astype(f32)
    for r in reciprocals(s):
        assert (F.e2m1_encode(side_of_quotient(x, s, r)) == exact_codes(x, s)).all()
    a = np.exp2(rng.uniform(-12, 12, 1_000_000)).astype(f32)
    assert (F.e4m3_encode(side_of_quotient(a, np.full_like(a, f32(6.0)), np.full_like(a, f32(0.16666667))))
            == exact_scale(a)).all()


def test_the_residual_is_exact():
    # what the second fma is given: x - y s, without a rounding
    x, s = near_borders(range(-40, 41))
    s = s.astype(f32)
    for r in reciprocals(s):
        y = kept12((x * r).astype(f32))
        assert (fma(-y, s, x).astype(np.float64) == x.astype(np.float64) - y.astype(np.float64) * s).all()


def test_short_sources_need_no_residual():
    # all bf16 from 2^-8 to 8 of every scale (a code's borders begin at 1/4): one product rounded to 12 bits
    m = np.arange(128, 256, dtype=np.float64) / 128
    e = np.floor(np.log2(SCALES))[:, None, None] + np.arange(-9, 4)[:, None]
    x = (m * np.exp2(e)).reshape(len(SCALES), -1)
    keep = x <= 8 * SCALES[:, None]
    x = np.where(keep, x, SCALES[:, None]).astype(f32)               # (a scale has four bits: bf16 too)
    s = np.broadcast_to(SCALES[:, None], x.shape)
    want = exact_codes(x, s)
    on = (x.astype(np.float64)[..., None] == BORDERS * s[..., None]).any(-1)
    assert on.sum() >= 7 * len(SCALES)                                # every border itself is among them
    for r in reciprocals(s.astype(f32)):
        y = kept12((x * r).astype(f32))
        assert (F.e2m1_encode(y) == want).all()
        # and without the rounding some would not be
    assert sum((F.e2m1_encode((x * r).astype(f32)) != want).sum() for r in reciprocals(s.astype(f32))) > 0


def test_the_gap_of_short_sources():
    # |x| / (t s) is 1 or at least 2^-8 away from it: odd parts X < 256 of x, T = 1, 3, 5 or 7 of t and S < 16 of s
    X, T, S = np.arange(1, 256), np.array([1, 3, 5, 7]), np.arange(1, 16)
    ts = np.unique(T[:, None] * S)
    q = X[:, None, None] * np.exp2(np.arange(-9, 10)) / ts[:, None]
    gap = np.abs(q - 1)
    assert ts.max() == 105 and gap[gap > 0].min() >= 2.0 ** -8


def test_the_restated_fma_rounds_once():
    from fractions import Fraction
    rng = np.random.default_rng(7)
    # products of 24 bits and sums that lie on, just beside and off a tie of binary32
    a = rng.integers(1 << 23, 1 << 24, 4000).astype(f32)
    b = np.exp2(rng.integers(-60, -20, 4000)).astype(f32) * rng.choice([1.0, -1.0, 1 + 2.0 ** -23], 4000).astype(f32)
    c = rng.integers(1 << 23, 1 << 24, 4000).astype(f32) * np.exp2(rng.integers(-30, 1, 4000)).astype(f32)
    a[:1000], b[:1000], c[:1000] = f32(2.0 ** -24), f32(1.0), f32(1.0)
    b[250:500], b[500:750], c[750:1000] = f32(1 + 2.0 ** -23), f32(1 - 2.0 ** -24), f32(1 + 2.0 ** -23)
    got = fma(a, b, c)
    for x, y, z, g in zip(a, b, c, got):
        exact = Fraction(float(x)) * Fraction(float(y)) + Fraction(float(z))
        err = abs(Fraction(float(g)) - exact)
        for n in (np.nextafter(g, f32(np.inf)), np.nextafter(g, f32(-np.inf))):
            far = abs(Fraction(float(n)) - exact)
            assert err < far or (err == far and int(g.view(np.int32)) % 2 == 0)
