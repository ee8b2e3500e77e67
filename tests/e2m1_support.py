"""Helpers of the E2M1 cache tests."""

import numpy as np
import torch

from oracle import chunk as OC
from oracle import formats as F
from oracle import paged_attention as PA

from .gpu_support import bits16


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


def chunk_case(q_lens, ctxs, H_q, H_kv, D, bs, scaled=True, softcap=0.0, window=0, bias=False, prefix=None, seed=1,
               spare=5, tail_rows=0, q_mult=1.0, free_behind_window=False):
    """A case of the ragged-chunk tests (chunk_support.device_args takes it) over
    E2M1 caches: NaN scales and any codes in every slot no sequence holds."""
    gen = torch.Generator().manual_seed(seed)
    B = len(q_lens)
    nblk = [-(-c // bs) for c in ctxs]
    mb = max(max(nblk, default=0), 1)
    n = sum(nblk) + spare
    perm = torch.randperm(n, generator=gen).tolist()
    table = np.full((B, mb), -1, dtype=np.int32)
    k = 0
    for b in range(B):
        table[b, :nblk[b]] = perm[k:k + nblk[b]]
        k += nblk[b]
    owned = np.zeros((n, bs), dtype=bool)
    for b in range(B):
        see = OC.visible(ctxs[b], q_lens[b], window, 0 if prefix is None else prefix[b]).any(axis=0)
        for j in range(nblk[b]):
            m = min(bs, ctxs[b] - j * bs)
            if free_behind_window and not see[j * bs:j * bs + m].any():
                table[b, j] = -1
            else:
                owned[table[b, j], :m] = True
    values, bytes_ = [], []
    for _ in range(2):
        codes, sc = F.e2m1_unpack(pool(gen, n, H_kv, bs, D).numpy())
        values.append(F.e2m1_values(F.e2m1_pack(codes, sc)))
        bad = np.broadcast_to(~owned[:, None, :], (n, H_kv, bs))
        sc = sc.copy()
        sc[bad] = 0x7F
        bytes_.append(torch.from_numpy(F.e2m1_pack(codes, sc)))
    ks = vs = None
    if scaled:
        ks, vs = (0.5 + torch.rand((B, H_kv), generator=gen) for _ in range(2))
    starts = np.concatenate([[0], np.cumsum(q_lens)]).astype(np.int32)
    q = (torch.randn((int(starts[-1]) + tail_rows, H_q, D), generator=gen) * q_mult).to(torch.bfloat16)
    slopes = torch.exp2(-8.0 * torch.arange(1, H_q + 1) / H_q).float() if bias else None
    return dict(q=q, kc=bytes_[0], vc=bytes_[1], kval=values[0], vval=values[1], table=table,
                ctx=np.array(ctxs, dtype=np.int32), starts=starts, scale=D ** -0.5, softcap=softcap, window=window,
                slopes=slopes, prefix=prefix, ks=ks, vs=vs, max_q=max(max(q_lens, default=1), 1),
                max_ctx=max(max(ctxs, default=1), 1))


def chunk_want(case):
    """(oracle, bound on the error of a right kernel), float64 [T, H_q, D].

    The caches' values and their products with the groups' scales are exact in
    f16, as is q here.  The output is rounded once to bf16 (2^-8 of itself),
    every weight once to f16: 2^-11 of A = sum p |v| / sum p.  A score is a
    binary32 sum of D products, off by at most D 2^-23 sum |q k| scale: the
    larger channels bring that to 2^-16 x 40 here, which enters numerator and
    denominator: with the exponential's 2^-22 below 2^-9 of A.
    """
    ks = None if case["ks"] is None else case["ks"].numpy()
    vs = None if case["vs"] is None else case["vs"].numpy()
    args = (case["table"], case["ctx"], case["starts"], case["scale"], case["softcap"], case["window"],
            None if case["slopes"] is None else case["slopes"].numpy(), case["prefix"], ks, vs)
    q = bits16(case["q"])
    ref = OC.chunk_attention(q, case["kval"], case["vval"], PA.VALUES, *args)
    A = OC.chunk_attention(q, case["kval"], np.abs(case["vval"]), PA.VALUES, *args)
    S = np.zeros_like(ref)
    H, bs = case["vval"].shape[1:3]
    for b, ctx in enumerate(case["ctx"]):
        for h in range(H):
            v = PA.dequantize(PA.gather_sequence(case["vval"], np.maximum(case["table"][b], 0), int(ctx), h, bs),
                              PA.VALUES, None if vs is None else vs[b, h])
            G = ref.shape[1] // H
            S[case["starts"][b]:case["starts"][b + 1], h * G:(h + 1) * G] = np.abs(v).sum(0)
    return ref, (2.0 ** -8 * np.abs(ref) * (1 + 2.0 ** -7) + (2.0 ** -11 + 2.0 ** -9) * A + 2.0 ** -25 * S + 1e-30)


def chunk_check(out, case, ref=None, tol=None):
    if ref is None:
        ref, tol = chunk_want(case)
    got = F.bf16_bits_to_f64(bits16(out))
    rows = ~np.isnan(ref[:, 0, 0])
    assert np.isfinite(got[rows]).all()
    err = np.abs(got[rows] - ref[rows])
    worst = float((err / tol[rows]).max()) if err.size else 0.0
    assert worst <= 1.0, f"error {worst:.2f} of the bound"
