"""Cases and tolerances of the ragged-chunk attention tests."""

import numpy as np
import torch

from oracle import chunk as OC
from oracle import formats as F
from oracle import paged_attention as PA

from .gpu_support import BF16_NAN, E4M3_NAN, bits16


def make_case(q_lens, ctxs, H_q, H_kv, D, bs, kv="bf16", softcap=0.0, window=0, bias=False, prefix=None, seed=1,
              spare=5, tail_rows=0, q_mult=1.0, free_behind_window=False):
    """Paged caches that hold each sequence's ctx tokens, over a shuffled pool,
    NaN in every slot no sequence holds; `tail_rows` rows of q past the last
    sequence; with `free_behind_window`, blocks no new token sees are gone (-1
    in the table, NaN in the pool)."""
    gen = torch.Generator().manual_seed(seed)
    B = len(q_lens)
    nblk = [-(-c // bs) for c in ctxs]
    mb = max(max(nblk, default=0), 1)
    pool = sum(nblk) + spare
    perm = torch.randperm(pool, generator=gen).tolist()
    table = np.full((B, mb), -1, dtype=np.int32)
    k = 0
    for b in range(B):
        table[b, :nblk[b]] = perm[k:k + nblk[b]]
        k += nblk[b]
    shape = (pool, H_kv, bs, D)
    if kv == "bf16":
        kc, vc = (torch.randn(shape, generator=gen).to(torch.bfloat16) for _ in range(2))
        kraw, vraw, nan = kc.view(torch.int16), vc.view(torch.int16), int(np.int16(BF16_NAN))
        ks = vs = None
    else:
        kc, vc = ((torch.randn(shape, generator=gen) * 64).to(torch.float8_e4m3fn).view(torch.uint8)
                  for _ in range(2))
        kraw, vraw, nan = kc, vc, E4M3_NAN
        ks, vs = ((0.5 + torch.rand((B, H_kv), generator=gen)) / 64 for _ in range(2))
    owned = np.zeros((pool, bs), dtype=bool)
    for b in range(B):
        see = OC.visible(ctxs[b], q_lens[b], window, 0 if prefix is None else prefix[b]).any(axis=0)
        for j in range(nblk[b]):
            n = min(bs, ctxs[b] - j * bs)
            if free_behind_window and not see[j * bs:j * bs + n].any():
                table[b, j] = -1
            else:
                owned[table[b, j], :n] = True
    bad = torch.from_numpy(~owned)
    kraw.permute(0, 2, 1, 3)[bad] = nan
    vraw.permute(0, 2, 1, 3)[bad] = nan
    starts = np.concatenate([[0], np.cumsum(q_lens)]).astype(np.int32)
    q = (torch.randn((int(starts[-1]) + tail_rows, H_q, D), generator=gen) * q_mult).to(torch.bfloat16)
    slopes = torch.exp2(-8.0 * torch.arange(1, H_q + 1) / H_q).float() if bias else None
    return dict(q=q, kc=kc, vc=vc, table=table, ctx=np.array(ctxs, dtype=np.int32), starts=starts, scale=D ** -0.5,
                softcap=softcap, window=window, slopes=slopes, prefix=prefix, ks=ks, vs=vs, kv=kv,
                max_q=max(max(q_lens, default=1), 1), max_ctx=max(max(ctxs, default=1), 1))


def device_args(case, dev):
    """(positional, keyword) arguments of pkv.chunk_attention."""
    def up(x):
        return None if x is None else (torch.as_tensor(x) if not torch.is_tensor(x) else x).to(dev)
    prefix = None if case["prefix"] is None else torch.tensor(case["prefix"], dtype=torch.int32)
    return ((up(case["q"]), up(case["kc"]), up(case["vc"]), up(case["table"]), up(case["ctx"]), up(case["starts"]),
             case["scale"]),
            dict(max_q_len=case["max_q"], max_context_len=case["max_ctx"], k_scale=up(case["ks"]),
                 v_scale=up(case["vs"]), softcap=case["softcap"], window=case["window"], slopes=up(case["slopes"]),
                 prefix_lens=up(prefix)))


def want(case):
    """(oracle, bound on the error of a right kernel), float64 [T, H_q, D].

    The output is rounded once to bf16 (2^-8 of itself), every weight once to
    the products' 16-bit type (2^-8 for bf16, 2^-11 for f16), which moves the
    output by at most that share of A = sum p |v| / sum p.  A score is a
    binary32 sum of D products, off by at most D 2^-23 sum |q k| scale, about
    2^-16 x 8 here, and enters numerator and denominator: with the
    exponential's 2^-22 well below 2^-10 of A.
    """
    ks = None if case["ks"] is None else case["ks"].numpy()
    vs = None if case["vs"] is None else case["vs"].numpy()
    if case["kv"] == "bf16":
        kc, vc, dt, eps = bits16(case["kc"]), bits16(case["vc"]), PA.BF16, 2.0 ** -8
        vabs = vc & 0x7FFF
    else:
        kc, vc, dt, eps = case["kc"].numpy(), case["vc"].numpy(), PA.E4M3, 2.0 ** -11
        vabs = vc & 0x7F
    args = (case["table"], case["ctx"], case["starts"], case["scale"], case["softcap"], case["window"],
            None if case["slopes"] is None else case["slopes"].numpy(), case["prefix"], ks, vs)
    ref = OC.chunk_attention(bits16(case["q"]), kc, vc, dt, *args)
    A = OC.chunk_attention(bits16(case["q"]), kc, vabs, dt, *args)
    return ref, 2.0 ** -8 * np.abs(ref) * (1 + 2.0 ** -7) + (eps + 2.0 ** -10) * A + 1e-30


def check(out, case, ref=None, tol=None):
    if ref is None:
        ref, tol = want(case)
    got = F.bf16_bits_to_f64(bits16(out))
    rows = ~np.isnan(ref[:, 0, 0])
    assert np.isfinite(got[rows]).all()
    err = np.abs(got[rows] - ref[rows])
    worst = float((err / tol[rows]).max()) if err.size else 0.0
    assert worst <= 1.0, f"error {worst:.2f} of the bound"
