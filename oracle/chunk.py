"""Ragged chunk attention, rotary positions and token compaction in float64.

TEST INFRASTRUCTURE ONLY (see the package docstring).

Attention: query i of the n new tokens of a sequence of ctx tokens sits at
pos = ctx - n + i; its score against key t is z = scale q.k, capped to
cap * tanh(z / cap), plus slope * (t - pos); it sees key t < ctx iff
t < prefix or pos - window < t <= pos; the output is softmax(z) V, zeros for
a query that sees nothing ([SC] "9. Failure modes and limitations", item 3,
and "4. Internal workings", step 4, with the scores as models define them).

Rotary positions: pair (x1, x2) of a head's first rotary elements is the
complex number x1 + i x2, times magnitude * e^(i pos f).
"""

import numpy as np

from .formats import bf16_bits_to_f64
from .paged_attention import dequantize, gather_sequence


def visible(ctx, n, window=0, prefix=0):
    """bool [n, ctx]: which keys each new token sees."""
    t = np.arange(ctx)[None, :]
    pos = (ctx - n + np.arange(n))[:, None]
    see = t <= pos
    if window > 0:
        see &= t > pos - window
    see |= t < prefix
    return see & (pos >= 0)


def chunk_attention(q_bits, k_cache, v_cache, cache_dtype, block_tables, context_lens, q_starts, scale,
                    softcap=0.0, window=0, slopes=None, prefix_lens=None, k_scale=None, v_scale=None):
    """float64 [T, H_q, D]; rows of no sequence stay NaN."""
    q = bf16_bits_to_f64(q_bits)
    T, H_q, D = q.shape
    H_kv, bs = k_cache.shape[1], k_cache.shape[2]
    G = H_q // H_kv
    out = np.full((T, H_q, D), np.nan)
    for b in range(len(context_lens)):
        lo, hi, ctx = int(q_starts[b]), int(q_starts[b + 1]), int(context_lens[b])
        n = hi - lo
        if n == 0:
            continue
        prefix = 0 if prefix_lens is None else min(max(int(prefix_lens[b]), 0), ctx)
        see = visible(ctx, n, window, prefix)
        some = see.any(axis=1)
        pos = ctx - n + np.arange(n)
        away = (np.arange(ctx)[None, :] - pos[:, None]).astype(np.float64)
        # a table need not name blocks that no query sees
        table = np.maximum(np.asarray(block_tables[b]), 0)
        used = see.any(axis=0)
        for h in range(H_kv):
            ks = None if k_scale is None else k_scale[b, h]
            vs = None if v_scale is None else v_scale[b, h]
            K = dequantize(gather_sequence(k_cache, table, ctx, h, bs), cache_dtype, ks)
            V = dequantize(gather_sequence(v_cache, table, ctx, h, bs), cache_dtype, vs)
            K, V = np.where(used[:, None], K, 0.0), np.where(used[:, None], V, 0.0)
            for hq in range(h * G, (h + 1) * G):
                z = scale * (q[lo:hi, hq] @ K.T)
                if softcap > 0:
                    z = softcap * np.tanh(z / softcap)
                if slopes is not None:
                    z = z + float(slopes[hq]) * away
                z = np.where(see, z, -np.inf)
                o = np.zeros((n, D))
                if some.any():
                    zs = z[some]
                    p = np.exp(zs - zs.max(axis=1, keepdims=True))
                    o[some] = (p / p.sum(axis=1, keepdims=True)) @ V
                out[lo:hi, hq] = o
    return out


def rotate(x, positions, inv_freq, interleaved=False, magnitude=1.0):
    """x [N, H, D] float64 with its first 2 * len(inv_freq) elements turned."""
    half = len(inv_freq)
    rd = 2 * half
    angle = np.asarray(positions, dtype=np.float64)[:, None] * np.asarray(inv_freq, dtype=np.float64)[None, :]
    z = magnitude * np.exp(1j * angle)[:, None, :]
    y = np.array(x, dtype=np.float64)
    if interleaved:
        a, b = slice(0, rd, 2), slice(1, rd, 2)
    else:
        a, b = slice(0, half), slice(half, rd)
    w = (y[..., a] + 1j * y[..., b]) * z
    y[..., a], y[..., b] = w.real, w.imag
    return y


def compact(cache, block_tables, keep, keep_starts, dst_start=None):
    """`cache` [NB, H, bs, D] with every kept row moved, all read before any is written."""
    bs = cache.shape[2]
    new = cache.copy()
    for b in range(len(keep_starts) - 1):
        first = 0 if dst_start is None else int(dst_start[b])
        for j, s in enumerate(keep[keep_starts[b]:keep_starts[b + 1]]):
            d = first + j
            new[block_tables[b][d // bs], :, d % bs] = cache[block_tables[b][s // bs], :, s % bs]
    return new
