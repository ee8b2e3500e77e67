"""Caps at the ends of binary32 and of the two ways they are computed."""

import numpy as np
import pytest
import torch

import paged_kv_cache_222_gb300 as pkv

from . import chunk_support as C

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda", 0)

FEW = ([1, 2], [300, 65])            # rows of the mma.sync kernel
MANY = ([40, 3, 200], [300, 65, 211])  # of the tcgen05 kernel


def run(case, **kw):
    args, kwargs = C.device_args(case, DEV)
    kwargs.update(kw)
    out = pkv.chunk_attention(*args, **kwargs)
    assert pkv.device_error(DEV) == 0
    return out


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("softcap", [1e-8, 1e-9, 1e-11, 1e-16, 1e-24, 1e-33])
@pytest.mark.parametrize("lens", [FEW, MANY], ids=["few", "many"])
def test_products_of_zero_under_tiny_caps(lens, softcap, D, bias, kv):
    # a query row of zeros has capped scores of 0: the mean of its visible values
    # (with a bias: weighted by distance)
    case = C.make_case(*lens, 8, 2, D, 16, kv, softcap=softcap, bias=bias, seed=79)
    case["q"][0] = 0
    case["q"][1, 3] = 0
    C.check(run(case), case)


def spread_case(lens, softcap, H_q, H_kv, D, bs, kv, seed):
    """Scores anywhere between far below and far above the cap, row by row, a
    third of the rows around 0.35 of it.  Key t has three elements: 256 and 1,
    which with the query's fix the row's score to a fraction of a unit, and an
    offset that spreads the keys over +- 1 unit after the cap's slope (at most
    16 before it); the offset's sign is its value, in every element.  All else
    is 0, so that products and their sums are exact in binary32 or nearly, and
    what an output is off by is what the capped scores are."""
    case = C.make_case(*lens, H_q, H_kv, D, bs, kv, softcap=softcap, seed=seed)
    g = torch.Generator().manual_seed(seed + 1)
    T = case["q"].shape[0]

    def wide(c):
        return c.float() if kv == "bf16" else c.view(torch.float8_e4m3fn).float()

    def narrow(c):
        return c.to(torch.bfloat16) if kv == "bf16" else c.to(torch.float8_e4m3fn).view(torch.uint8)
    nan = torch.isnan(wide(case["kc"])[..., 0])
    off = torch.randint(-16, 17, nan.shape, generator=g) / 16.0
    kc = torch.zeros(nan.shape + (D,))
    kc[..., 3] = 256.0
    kc[..., 20] = 1.0
    kc[..., D - 2] = off
    vc = torch.where(off < 0, -1.0, 1.0)[..., None].repeat(1, 1, 1, D)
    kc[nan] = float("nan")
    vc[nan] = float("nan")
    case["kc"], case["vc"] = narrow(kc), narrow(vc)
    if kv != "bf16":
        case["ks"].fill_(1.0)
        case["vs"].fill_(1.0)
    # queries beside E4M3 caches are taken as f16: within its range
    case["scale"] = scale = 1.0 / 1024 if kv == "bf16" else softcap / 4096
    y = torch.exp(torch.empty((T, H_q), dtype=torch.float64).uniform_(np.log(0.02), np.log(3.0), generator=g))
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
      the weight's rounding for the products (2^-8, 2^-11), in the numerator
        alone: times sum p |v| = 1;
      twice 2^-22 for the exponential and the sums;
      a capped score c's error: up to 0.35 of the cap 2^-13 (the bound of the
        short polynomial) or 2^-21.7 c (the long one's 4.1e-8 and its five
        roundings), above 2^-22.2 of the cap (2 / (e^2y + 1), at most 0.66, with
        an exponential of 2^-22.5, a reciprocal of 2^-23 and two roundings),
        and 2^-23 c for the multipliers and the row maximum's subtraction.
    The output is rounded to bf16."""
    q = case["q"].double().numpy()
    cap = case["softcap"]
    z = case["scale"] * np.abs(q[..., 3] * 256.0 + q[..., 20])
    off = case["scale"] * np.abs(q[..., -2])
    c = cap * np.tanh((z + off) / cap)
    score = np.maximum(2.0 ** -13, 2.0 ** -21.7 * c) * (z - off <= 0.35 * cap)
    score = np.maximum(score, 2.0 ** -22.2 * cap * (z + off > 0.35 * cap)) + 2.0 ** -23 * c
    eps = 2.0 ** -8 if case["kv"] == "bf16" else 2.0 ** -11
    return eps + (2.0 ** -21 + score[..., None] * 1.01) * (1 - ref ** 2) + 2.0 ** -8 * np.abs(ref) * 1.01


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("softcap", [20.0, 60.0, 100.0, 101.0, 1000.0, 1e4, 1e5])
@pytest.mark.parametrize("lens", [FEW, MANY], ids=["few", "many"])
def test_scores_from_far_below_to_far_above_large_caps(lens, softcap, D, kv):
    case = spread_case(lens, softcap, 8, 2, D, 16, kv, seed=int(softcap) % 1000)
    ref, _ = C.want(case)
    C.check(run(case), case, ref, spread_bound(case, ref))
