"""Which E2M1 code a value has and which E4M3 scale a group, decided exactly.

A border is t s of a code's border t (1/4 ... 5) and a scale s, or 6 m of the
midpoint m of two E4M3 numbers: at most seven significant bits, so binary64
holds it and a comparison with a binary32 value is exact.
"""

import numpy as np

from oracle import formats as F

f32 = np.float32
SCALES = F.e4m3_to_f64(np.arange(1, 0x7F, dtype=np.uint8))          # every positive finite one
E4M3 = F.e4m3_to_f64(np.arange(0x7F, dtype=np.uint8))
BORDERS = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0])


def exact_codes(x, s):
    """Code of binary32 x over scale s > 0 (broadcast): the nearest magnitude, ties to even, the sign kept."""
    a, s = np.abs(x.astype(np.float64)), np.asarray(s, dtype=np.float64)
    code = sum(((a >= t * s) if i % 2 else (a > t * s)).astype(np.uint8) for i, t in enumerate(BORDERS))
    return code | (np.signbit(x).astype(np.uint8) << np.uint8(3))


def exact_scale(amax):
    """E4M3 code of a group's largest magnitude over 6, ties to even, saturating."""
    a = np.minimum(amax.astype(np.float64), 6 * 448.0)
    mid = 6.0 * (E4M3[1:] + E4M3[:-1]) / 2                           # past code i: code i + 1, at it the even one
    lo = np.searchsorted(mid, a, side="left")                        # midpoints below a
    hi = np.searchsorted(mid, a, side="right")
    return np.where(lo == hi, lo, lo + lo % 2).astype(np.uint8)      # (equal to midpoint lo: codes lo, lo + 1)


def around(v, steps):
    """Binary32 values `steps` last places from exactly representable v > 0, [..., len(steps)]."""
    bits = v.astype(f32).view(np.int32)[..., None] + np.asarray(steps, dtype=np.int32)
    return bits.astype(np.int32).view(f32)


def near_borders(steps=(-3, -2, -1, 0, 1, 2, 3)):
    """(values, scales): every border of every scale and its neighbours, both signs."""
    x = around(SCALES[:, None] * BORDERS, steps).reshape(len(SCALES), -1)
    x = np.concatenate([x, -x], axis=-1)
    return x, np.broadcast_to(SCALES[:, None], x.shape)
