"""The polynomials behind capped scores against tanh in 64 bits (host build of
the constants the kernels use)."""

import subprocess

import numpy as np
import pytest

from paged_kv_cache_222_gb300 import build as B

HARNESS = r"""
#include <cstdio>
#include "pkv_internal.h"
int main() {
  double cap;
  while (std::scanf("%lf", &cap) == 1) {
    float c[3], y_max;
    pkv::cap_coefficients(cap, c, y_max);
    std::printf("%.17g %.17g %.17g %.17g\n", c[0], c[1], c[2], y_max);
  }
  std::printf("%.17g %.17g %.17g %.17g\n", pkv::kCapC1, pkv::kCapC2, pkv::kCapC3, pkv::kCapLimit);
}
"""
CAPS = [1e-30, 1e-3, 1.0, 20.0, 50.0, 99.0, 100.0, 100.001, 101.0, 150.0, 300.0, 1e3, 1e4, 1e5, 1e6, 1e8]


@pytest.fixture(scope="module")
def values(tmp_path_factory):
    d = tmp_path_factory.mktemp("cap")
    (d / "cap.cu").write_text(HARNESS)
    subprocess.run([B.nvcc(), "-std=c++17", "-I", B.CSRC, "-I", B.INCLUDE, str(d / "cap.cu"), "-o", str(d / "cap")],
                   check=True, capture_output=True)
    out = subprocess.run([str(d / "cap")], input="\n".join(map(repr, CAPS)), check=True, capture_output=True,
                         text=True).stdout
    rows = [[float(x) for x in line.split()] for line in out.splitlines()]
    return dict(zip(CAPS, rows)), rows[-1]


def test_small_scores_are_off_by_less_than_a_fixed_amount(values):
    # whatever the cap: 2^-13 of a weight, next to its own rounding; the
    # coefficients' rounding to binary32 (2^-26) is of the score y^3 cap
    for cap, (c0, c1, c2, y_max) in values[0].items():
        y = np.linspace(0.0, y_max, 20001)
        t = y * y
        err = cap * np.abs(y * (c0 + c1 * t + c2 * t * t) - np.tanh(y))
        assert (err <= 2.0 ** -13 + 2.0 ** -25 * cap * y ** 3).all(), (cap, err.max())
        assert 0.35000001 >= y_max > 0.02


def test_ordinary_caps_hold_for_ordinary_scores(values):
    # the fast form takes scores up to 17 under a cap of 50, and at least 20 and
    # a growing number under larger ones
    ranges = [cap * v[3] for cap, v in values[0].items()]
    assert values[0][50.0][3] * 50.0 > 17
    assert all(a < b for a, b in zip(ranges, ranges[1:]) if a < 34)
    assert all(cap * v[3] >= 33 for cap, v in values[0].items() if cap >= 100)


def test_the_longer_polynomial_is_exact_to_binary32(values):
    c1, c2, c3, limit = values[1]
    assert limit == pytest.approx(0.35, rel=1e-7)
    y = np.linspace(1e-6, limit, 20001)
    t = y * y
    err = np.abs(y * (1 + t * (c1 + t * (c2 + t * c3))) / np.tanh(y) - 1)
    assert err.max() <= 4.2e-8
