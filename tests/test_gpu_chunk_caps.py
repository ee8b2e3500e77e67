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
