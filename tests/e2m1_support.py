"""Helpers of the E2M1 cache tests."""

import numpy as np
import torch

from oracle import formats as F


def token_bytes(cache):
    """(codes [tokens, H, D], scale codes [tokens, H, D / 16]) of a cache tensor, by flat slot."""
    codes, sc = F.e2m1_unpack(cache.cpu().numpy())
    return tuple(np.moveaxis(x, 1, 2).reshape((-1, x.shape[1], x.shape[3])) for x in (codes, sc))


def special_rows(D, seed=0):
    """Float32 rows [n, D] whose groups hold what rounding can go wrong on: ties
    of codes and of scales, saturation, scales that are subnormal or round to
    zero, zeros of both signs, infinities and NaN."""
    rng = np.random.default_rng(seed)
    rows = []
    ties = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0], dtype=np.float64)
    for e in range(-12, 10):                       # ties exactly at, just below and just above a scale of 2^e
        g = np.concatenate([ties, -ties]).astype(np.float32) * np.float32(2.0 ** e)
        up, down = np.nextafter(g, np.float32(np.inf)), np.nextafter(g, np.float32(-np.inf))
        for v in (g, np.where(np.abs(g) == 6 * 2.0 ** e, g, up), np.where(np.abs(g) == 6 * 2.0 ** e, g, down)):
            rows.append(v)
    for m in range(8):                             # every mantissa of a scale, and ties between two
        for s in ((8 + m) / 8, (8 + m + 0.5) / 8):
            g = (rng.uniform(-6, 6, 16) * s).astype(np.float32)
            g[3] = np.float32(6 * s)
            rows.append(g)
    for top in (0.0, 1e-45, 6 * 2.0 ** -10, np.nextafter(np.float32(6 * 2.0 ** -10), np.float32(1)), 6 * 2.0 ** -9,
                9 * 2.0 ** -9, 2688.0, 2689.0, 2784.0, 1e6, 3e38, np.inf):
        g = (rng.uniform(-1, 1, 16) * (top if np.isfinite(top) else 5e3)).astype(np.float32)
        g[5], g[6], g[7] = np.float32(top), np.float32(-top), np.float32(-0.0)
        rows.append(g)
    g = rng.standard_normal(16).astype(np.float32)
    g[9] = np.float32(np.nan)
    rows.append(g)
    per = D // 16
    while len(rows) % per:
        rows.append((rng.standard_normal(16) * 3).astype(np.float32))
    return np.concatenate(rows).reshape(-1, D)


def pool(gen, blocks, H, bs, D, loud=True):
    """A CPU cache tensor (uint8) of quantised normal values, some channels larger."""
    x = torch.randn((blocks, H, bs, D), generator=gen)
    if loud:
        x *= 1.0 + 7.0 * (torch.rand((H, 1, D), generator=gen) > 0.97)
    return torch.from_numpy(F.e2m1_pack(*F.e2m1_rows(x.numpy())))
