"""The polynomial for capped scores up to 1.25 caps (E2M1 caches, tcgen05)
against tanh in 64 bits: the constants that the kernel uses, in its own steps."""

import subprocess

import numpy as np
import pytest

from paged_kv_cache_222_gb300 import build as B

HARNESS = r"""
#include <cstdio>
#include "pkv_internal.h"
int main() {
  for (double x : {double(pkv::kMidC0), double(pkv::kMidC1), double(pkv::kMidC2), double(pkv::kMidC3),
                   double(pkv::kMidC4), double(pkv::kMidC5), double(pkv::kMidC6), double(pkv::kMidLimit),
                   pkv::kCapNear})
    std::printf("%.17g\n", x);
}
"""


@pytest.fixture(scope="module")
def values(tmp_path_factory):
    d = tmp_path_factory.mktemp("mid")
    (d / "mid.cu").write_text(HARNESS)
    subprocess.run([B.nvcc(), "-std=c++17", "-I", B.CSRC, "-I", B.INCLUDE, str(d / "mid.cu"), "-o", str(d / "mid")],
                   check=True, capture_output=True)
    out = subprocess.run([str(d / "mid")], check=True, capture_output=True, text=True).stdout
    return [float(x) for x in out.split()]


def steps(c, y, dt):
    """The kernel's: t = u u, a chain of fused multiply-adds, times u.  (A product of binary32 numbers is exact in
    binary64, so that each step rounds to binary32 as the fused one does.)"""
    u = y.astype(dt)
    t = (u * u).astype(dt).astype(np.float64)
    q = np.full_like(t, c[-1])
    for k in c[-2::-1]:
        q = (q * t + k).astype(dt).astype(np.float64)
    return u.astype(np.float64) * q if dt == np.float64 else (u * q.astype(dt)).astype(dt).astype(np.float64)


@pytest.mark.parametrize("dt,most", [(np.float64, 3.5e-7), (np.float32, 4.4e-7)])
def test_off_by_less_than_it_says(values, dt, most):
    c, limit = values[:7], values[7]
    assert limit == 1.25
    y = np.linspace(-limit, limit, 400_001).astype(np.float32).astype(np.float64)
    assert np.abs(steps(c, y, dt) - np.tanh(y)).max() < most


@pytest.mark.parametrize("i", range(7))
def test_every_coefficient_counts(values, i):
    c, y = list(values[:7]), np.linspace(0, values[7], 20_001)
    c[i] *= 1 + 2.0 ** -10
    assert np.abs(steps(c, y, np.float32) - np.tanh(y)).max() > 4.4e-7


def test_next_to_a_weights_own_rounding(values):
    assert values[8] == 100.0 and 4.4e-7 * values[8] < 2.0 ** -13


def test_a_hidden_score_stays_hidden(values):
    assert values[6] > 0
    with np.errstate(all="ignore"):
        for dt in (np.float32, np.float64):
            assert steps(values[:7], np.array([-np.inf]), dt)[0] == -np.inf
