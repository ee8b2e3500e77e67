"""Chunk attention over E2M1 caches on scores that are exact in binary32, so that
only the roundings an output is meant to have are left in the bound: peaked
weights, and capped scores on both sides of every way they are computed in."""

import numpy as np
import pytest
import torch

import paged_kv_cache_222_gb300 as pkv
from oracle import chunk as OC
from oracle import formats as F
from oracle import paged_attention as PA

from . import chunk_support as C
from . import e2m1_support as E
from .gpu_support import bits16

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda", 0)

SINGLE = ([1, 1, 1, 1, 1, 1], [1, 2, 17, 64, 65, 1000])
FEW = ([2, 1, 0, 2, 1, 2, 2, 1], [2, 1, 40, 33, 31, 32, 300, 129])
RAGGED = ([1, 5, 0, 33, 130, 64, 2], [1, 5, 40, 33, 300, 900, 257])
PROMPTS = ([1, 127, 128, 129, 300], [1, 127, 128, 129, 300])
LENS = pytest.mark.parametrize("lens", [SINGLE, FEW, RAGGED, PROMPTS], ids=["single", "few", "ragged", "prompts"])


def run(case, **kw):
    args, kwargs = C.device_args(case, DEV)
    kwargs.update(kw)
    out = pkv.chunk_attention(*args, **kwargs)
    assert pkv.device_error(DEV) == 0
    return out


def rewrite(case, name, codes_of, scale_code):
    """The cache's codes and scales replaced in the slots that sequences hold (the others keep NaN scales)."""
    codes, sc = F.e2m1_unpack(case[name].numpy())
    bad = sc == 0x7F
    codes = codes_of(codes.shape)
    sc = np.broadcast_to(scale_code, sc.shape)
    case["kval" if name == "kc" else "vval"] = F.e2m1_values(F.e2m1_pack(codes, sc))
    case[name] = torch.from_numpy(F.e2m1_pack(codes, np.where(bad, 0x7F, sc).astype(np.uint8)))


def oracle(case, v):
    args = (case["table"], case["ctx"], case["starts"], case["scale"], case["softcap"], case["window"],
            None if case["slopes"] is None else case["slopes"].numpy(), case["prefix"],
            None if case["ks"] is None else case["ks"].numpy(), None if case["vs"] is None else case["vs"].numpy())
    return OC.chunk_attention(bits16(case["q"]), case["kval"], v, PA.VALUES, *args)


@pytest.mark.parametrize("H_q,H_kv,D,bs", [(8, 2, 128, 16), (7, 1, 64, 32), (16, 1, 128, 32), (6, 3, 64, 16)])
@pytest.mark.parametrize("mods", [{}, dict(window=100), dict(split_tokens=128)], ids=["plain", "window", "splits"])
@LENS
def test_peaked_weights(lens, mods, H_q, H_kv, D, bs):
    """Queries of whole numbers up to 4 and keys of quarters up to 3/2: a product
    of a row is a whole number of quarters, below 2^10, so that binary32 sums of
    them in any order are exact, and the scores are far apart (of 128-wide heads
    by 15 units and more), a few weights holding a row.

    Of such a row: the weight's rounding to f16 (2^-11 of A = sum p |v| / sum p,
    2^-25 of the largest below 2^-14), its exponent (five roundings, 2^-24 each, of
    a score of at most Z, and 2^-22 for the exponential, entering numerator and
    denominator), sums of up to 1000 products (2^-14 of A each), the output's
    rounding to bf16 (2^-8).
    """
    case = E.chunk_case(*lens, H_q, H_kv, D, bs, seed=31 + D + bs, window=mods.get("window", 0))
    rng = np.random.default_rng(H_q)
    # codes 0..3 (0, 1/2, 1, 3/2), a scale of 1/2 or 1 for each group
    low = lambda shape: (rng.integers(0, 4, shape) | rng.integers(0, 2, shape) << 3).astype(np.uint8)
    rewrite(case, "kc", low, rng.choice([0x30, 0x38], D // 16).astype(np.uint8))
    case["q"] = torch.from_numpy(rng.integers(-4, 5, case["q"].shape).astype(np.float32)).bfloat16()
    case["scale"] = 0.5
    ref, A = oracle(case, case["vval"]), oracle(case, np.abs(case["vval"]))
    Z = 0.5 * float(case["ks"].max()) * 4 * 1.5 * D
    S = np.zeros_like(ref)
    G = H_q // H_kv
    for b, ctx in enumerate(case["ctx"]):
        for h in range(H_kv):
            v = PA.dequantize(PA.gather_sequence(case["vval"], np.maximum(case["table"][b], 0), int(ctx), h, bs), PA.VALUES,
                              case["vs"].numpy()[b, h])
            S[case["starts"][b]:case["starts"][b + 1], h * G:(h + 1) * G] = np.abs(v).sum(0)
    tol = (2.0 ** -8 * np.abs(ref) * (1 + 2.0 ** -7) + (2.0 ** -11 + 2.0 ** -13 + 2 * (5 * 2.0 ** -24 * Z + 2.0 ** -22)) * A
           + 2.0 ** -25 * S + 1e-30)
    E.chunk_check(run(case, **{k: v for k, v in mods.items() if k == "split_tokens"}), case, ref, tol)


def spread(lens, softcap, reach, H_q, H_kv, D, bs, bias, seed):
    """Scores of up to `reach` caps, row by row, a third of the rows around 0.35
    of the cap.  Key t has three elements: 256 and 1, which with the query's fix
    the row's score to a fraction of a unit, and an offset of up to 3/4 that
    spreads the keys over +- 3/4 of a unit after the cap's slope (at most 16 before
    it); the offset's sign is its value, in every element.  All else is 0, so that
    products and their sums are exact in binary32 or nearly."""
    case = E.chunk_case(*lens, H_q, H_kv, D, bs, softcap=softcap, bias=bias, seed=seed, scaled=False)
    g = torch.Generator().manual_seed(seed + 1)
    off = torch.randint(-7, 8, case["kc"].shape[:3], generator=g).numpy()  # a code of the last group, scale 1/8
    def keys(shape):
        c = np.zeros(shape, dtype=np.uint8)
        c[..., 3] = 6                                                 # 4, of a group of scale 64
        c[..., 20] = 2                                                # 1, of a group of scale 1
        c[..., D - 2] = np.abs(off) | (off < 0) * 8
        return c
    sc = np.full(D // 16, 0x38, dtype=np.uint8)
    sc[0], sc[-1] = 0x68, 0x20
    assert F.e4m3_to_f64(sc[[0, 1, -1]]).tolist() == [64.0, 1.0, 0.125]
    rewrite(case, "kc", keys, sc)
    rewrite(case, "vc", lambda shape: np.where(off < 0, 10, 2).astype(np.uint8)[..., None].repeat(D, -1), np.uint8(0x38))
    T = case["q"].shape[0]
    case["scale"] = scale = softcap / 4096                            # (queries are taken as f16: within its range)
    y = torch.exp(torch.empty((T, H_q), dtype=torch.float64).uniform_(np.log(0.02), np.log(reach), generator=g))
    y[::3] = 0.35 + (torch.rand(y[::3].shape, generator=g, dtype=torch.float64) - 0.5) * 2.0 / softcap
    sign = torch.where(torch.rand((T, H_q), generator=g) < 0.3, -1.0, 1.0).double()
    z = sign * y * softcap / scale
    q = torch.zeros((T, H_q, D), dtype=torch.bfloat16)
    q[..., 3] = (z / 256.0).to(torch.bfloat16)
    q[..., 20] = (z - q[..., 3].double() * 256.0).to(torch.bfloat16)
    q[..., D - 2] = (torch.cosh(y) ** 2).clamp(max=16.0).div(scale).to(torch.bfloat16)
    case["q"] = q
    return case


def spread_bound(case, ref):
    """Values are +- 1, so with weights off by a factor of up to 1 + e each the
    output moves by at most e sum p |v - out| = e (1 - out^2).  e is
      the weight's rounding for the products (2^-11), in the numerator alone:
        times sum p |v| = 1;
      twice 2^-22 for the exponential and the sums;
      a capped score c's error: up to 0.35 of the cap 2^-13 (the bound of the
        short polynomial), above 4.4e-7 of the cap (the longer one's, which is more
        than 2 / (e^2y + 1)'s 2^-22.2), and 2^-23 c for the multipliers and the
        row maximum's subtraction; twice 2^-24 of the bias.
    The output is rounded to bf16."""
    q = case["q"].double().numpy()
    cap = case["softcap"]
    z = case["scale"] * np.abs(q[..., 3] * 256.0 + q[..., 20])
    off = 0.75 * case["scale"] * np.abs(q[..., -2])
    c = cap * np.tanh((z + off) / cap)
    score = np.maximum(2.0 ** -13 * (z - off <= 0.35 * cap), 4.4e-7 * cap * (z + off > 0.35 * cap)) + 2.0 ** -23 * c
    if case["slopes"] is not None:
        score = score + 2.0 ** -23 * case["slopes"].double().numpy() * case["max_ctx"]
    return 2.0 ** -11 + (2.0 ** -21 + score[..., None] * 1.01) * (1 - ref ** 2) + 2.0 ** -8 * np.abs(ref) * 1.01


@pytest.mark.parametrize("H_q,H_kv,D,bs", [(8, 2, 128, 16), (7, 1, 64, 32)])
@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("reach", [0.3, 1.2, 3.0])
@pytest.mark.parametrize("softcap", [20.0, 60.0, 100.0])
@pytest.mark.parametrize("lens", [([1, 2], [300, 65]), ([40, 3, 200], [300, 65, 211])], ids=["few", "many"])
def test_capped_scores_in_every_way(lens, softcap, reach, bias, H_q, H_kv, D, bs):
    case = spread(lens, softcap, reach, H_q, H_kv, D, bs, bias, seed=int(softcap) + int(10 * reach))
    ref = oracle(case, case["vval"])
    E.chunk_check(run(case), case, ref, spread_bound(case, ref))
