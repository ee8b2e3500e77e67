"""The stated bound on rotary angles, at positions where the angle returns
almost to a whole turn: there the sine is small, and its bf16 value resolves
the angle's error."""

import math
from fractions import Fraction

import numpy as np
import pytest
import torch

import paged_kv_cache_222_gb300 as pkv

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda", 0)
# pi to 80 decimals
PI = Fraction(31415926535897932384626433832795028841971693993751058209749445923078164062862090, 10 ** 79)


def near_turns(f, limit):
    """Positions up to `limit` whose angle pos * f is nearest to whole turns: the
    denominators of f / 2 pi's continued fraction, largest last."""
    x = Fraction(f) / (2 * PI)
    x -= math.floor(x)
    p0, q0, p1, q1, r, out = 0, 1, 1, 0, x, []
    while True:
        a = math.floor(r)
        p0, q0, p1, q1 = p1, q1, a * p1 + p0, a * q1 + q0
        if q1 > limit:
            return out
        out.append(q1)
        if r == a:
            return out
        r = 1 / (r - a)


@pytest.mark.parametrize("limit", [2 ** 20, 2 ** 31, 2 ** 40])
@pytest.mark.parametrize("interleaved", [False, True])
def test_angles_at_far_positions(limit, interleaved):
    D, rd = 64, 32
    f = pkv.rotary_frequencies(rd, 10000.0)
    f[0] = 0.7310585786300049
    pos = []
    for i in (0, 1, 3, 7):
        pos += [s * n for n in near_turns(float(f[i]), limit)[-6:] for s in (1, -1)]
    pos += [limit, -limit, limit - 1]
    n = len(pos)
    x = torch.zeros((n, 1, D), dtype=torch.float32, device=DEV)
    cos_at = list(range(0, rd, 2)) if interleaved else list(range(rd // 2))
    sin_at = list(range(1, rd, 2)) if interleaved else list(range(rd // 2, rd))
    x[:, 0, cos_at] = 1.0                       # every pair (1, 0): turned to (cos, sin)
    kc = torch.zeros((n // 16 + 1, 1, 16, D), dtype=torch.bfloat16, device=DEV)
    slots = torch.arange(n, device=DEV)
    out = pkv.rotary_append(x, x, x, torch.tensor(pos, device=DEV), f.to(DEV), slots, kc, kc.clone(),
                            interleaved=interleaved)
    assert pkv.device_error(DEV) == 0
    got = out[:, 0].double().cpu().numpy()
    small = 0
    for r, p in enumerate(pos):
        for i in range(rd // 2):
            turns = Fraction(p) * Fraction(float(f[i])) / (2 * PI)
            turns -= round(turns)
            angle = float(turns * 2 * PI)
            bound = abs(p * float(f[i])) * 2.0 ** -52 + abs(p) * 2.0 ** -62 + 2.0 ** -22
            for at, want in ((cos_at[i], math.cos(angle)), (sin_at[i], math.sin(angle))):
                # rounded to bf16 after sine or cosine's own 2^-23
                assert abs(got[r, at] - want) <= (bound + 2.0 ** -23) * 1.01 + 2.0 ** -8 * (abs(want) + bound), (p, i)
            small += abs(angle) < 2.0 ** -12
    assert small >= 8                           # some really resolve it
    assert np.isfinite(got).all()
