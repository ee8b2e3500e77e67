"""More sequences than one warp has lanes (the tcgen05 kernel then finds a
unit's sequence by search) with everything a score can be, and scales that all
sequences share."""

import numpy as np
import pytest
import torch

import paged_kv_cache_222_gb300 as pkv

from . import chunk_support as C

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda", 0)


def run(case, **kw):
    args, kwargs = C.device_args(case, DEV)
    kwargs.update(kw)
    out = pkv.chunk_attention(*args, **kwargs)
    assert pkv.device_error(DEV) == 0
    return out


def ragged(B, seed, longest=90):
    rng = np.random.default_rng(seed)
    q = rng.integers(0, longest, B)
    q[rng.random(B) < 0.2] = 1
    q[rng.random(B) < 0.1] = 0
    ctx = q + rng.integers(0, 700, B)
    ctx[3] = max(0, int(q[3]) - 5)               # a context shorter than its new tokens
    return q.tolist(), ctx.tolist()


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("mods", [dict(window=100), dict(prefix=True), dict(window=65, prefix=True),
                                  dict(window=65, prefix=True, bias=True, softcap=20.0), dict(window=129, softcap=300.0)],
                         ids=["window", "prefix", "both", "all", "window+far cap"])
@pytest.mark.parametrize("B", [32, 33, 45, 70])
def test_many_sequences_windows_prefixes_and_splits(B, mods, D, kv):
    q, ctx = ragged(B, B)
    mods = dict(mods)
    if mods.pop("prefix", False):
        mods["prefix"] = [(i * 37) % 300 for i in range(B)]
    case = C.make_case(q, ctx, 8, 2, D, 16, kv, seed=B, **mods)
    ref, tol = C.want(case)
    for split in (0, 128, 384):
        C.check(run(case, split_tokens=split), case, ref, tol)


@pytest.mark.parametrize("lens", [([1] * 6, [1, 2, 17, 64, 65, 1000]), ([1, 5, 0, 33, 130, 64, 2], [1, 5, 40, 33, 300, 900, 257])],
                         ids=["single", "ragged"])
@pytest.mark.parametrize("D", [64, 128])
def test_scales_shared_by_all_sequences(lens, D):
    case = C.make_case(*lens, 8, 2, D, 16, "e4m3", seed=61)
    case["ks"][:] = case["ks"][0].clone()
    case["vs"][:] = case["vs"][0].clone()
    ref, tol = C.want(case)
    args, kw = C.device_args(case, DEV)
    per_row = pkv.chunk_attention(*args, **kw)
    kw.update(k_scale=kw["k_scale"][0].contiguous(), v_scale=kw["v_scale"][0].contiguous())
    shared = pkv.chunk_attention(*args, **kw)
    assert pkv.device_error(DEV) == 0
    C.check(shared, case, ref, tol)
    assert torch.equal(shared, per_row)


def test_rows_of_scales_further_apart():
    # a slice of wider rows of scales, by its row stride
    case = C.make_case([1, 40, 3], [300, 200, 77], 8, 2, 128, 16, "e4m3", seed=62)
    ref, tol = C.want(case)
    args, kw = C.device_args(case, DEV)
    wide = {}
    for name in ("k_scale", "v_scale"):
        w = torch.full((3, 5), float("nan"), device=DEV)
        w[:, :2] = kw[name]
        wide[name] = w.view(-1)
    out = pkv.chunk_attention(*args, **dict(kw, **wide, scale_row_stride=5))
    assert pkv.device_error(DEV) == 0
    C.check(out, case, ref, tol)
