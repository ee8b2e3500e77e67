"""Attention over E2M1 caches, what can be checked without a GPU: the plans'
splits against the kernels' own count of them, and what the C entry refuses."""

import ctypes

import numpy as np
import pytest

import paged_kv_cache_222_gb300 as pkv
from paged_kv_cache_222_gb300 import _lib as L
from paged_kv_cache_222_gb300 import build as B
from .test_chunk_host import chunk
from .test_chunk_splits_host import pieces

FAKE = ctypes.c_void_p(256)  # an aligned address: every call here is refused before it is read


@pytest.fixture(scope="module")
def lib():
    B.build()
    return L.load()


def desc(num_blocks=1 << 20, bs=16, H=2, D=128):
    return L.CacheDesc(num_blocks, bs, H, D, pkv.PKV_E2M1)


@pytest.mark.parametrize("bs,D", [(16, 128), (16, 64), (32, 128), (32, 64)])
@pytest.mark.parametrize("group", [1, 3, 8, 9, 16])
def test_pieces_fit_the_plan(lib, group, bs, D):
    # both kernels take 128 keys at a time
    rng = np.random.default_rng(group * 1000 + D + bs)
    c = desc(bs=bs, D=D)
    for _ in range(150):
        max_q = int(rng.choice([1, 1, 2, 5, 16, 17, 33, 257, 2000]))
        max_ctx = int(rng.choice([1, 127, 128, 129, 500, 1024, 3001, 9000, 40000]))
        window = int(rng.choice([0, 0, 1, 50, 127, 128, 129, 300, 5000]))
        has_prefix = bool(rng.random() < 0.4)
        split = int(rng.choice([0, 0, 128, 256, 640, 1024]))
        batch = int(rng.choice([1, 2, 7, 40]))
        T = int(rng.integers(max_q, max_q * batch + 1))
        p = pkv.chunk_plan(T, batch, max_q, 2 * group, c, max_ctx, window=window, has_prefix=has_prefix,
                           split_tokens=split)
        small = p.workers == 1
        assert small == (max_q * group <= 16)
        assert p.split_tokens % 128 == 0
        for _ in range(12):
            n = int(rng.integers(1, max_q + 1))
            ctx = int(rng.integers(0, max_ctx + 1)) if rng.random() < 0.8 else max_ctx
            prefix = int(rng.integers(0, max_ctx + 1)) if has_prefix else 0
            assert pieces(n, ctx, (16 if small else 256) // group, window, prefix, 128, p.split_tokens) <= p.max_splits


@pytest.mark.parametrize("kw", [{}, dict(D=64), dict(bs=32), dict(bs=32, D=64, H=1)])
@pytest.mark.parametrize("group", [1, 8, 9, 16])
def test_plans_of_single_tokens(lib, kw, group):
    c = desc(**kw)
    assert pkv.chunk_plan(0, 0, 1, group * c.num_kv_heads, c, 0).workspace_bytes == 0
    for batch in (1, 2, 3, 8, 17, 64, 300, 4000):
        for ctx in (1, 127, 128, 129, 1000, 1025, 2049, 8192, 30000, 200001, 1 << 21):
            p = pkv.chunk_plan(batch, batch, 1, group * c.num_kv_heads, c, ctx)
            assert p.workers == 1 and p.split_tokens % 128 == 0
            assert 128 <= p.split_tokens <= 1024 * c.block_size  # the ids that a CTA holds
            steps = -(-ctx // 128) * 128
            assert (p.max_splits - 1) * p.split_tokens < steps <= p.max_splits * p.split_tokens
            if p.max_splits > 1:
                assert p.workspace_bytes >= batch * group * c.num_kv_heads * p.max_splits * (c.head_dim + 2) * 4


@pytest.mark.parametrize("kw,ckw,code", [
    (dict(ks=FAKE), {}, 1),                                   # one of the two scales
    (dict(vs=FAKE), {}, 1),
    (dict(ks=FAKE, vs=FAKE, stride=-1), {}, 1),
    (dict(kc=ctypes.c_void_p(264)), {}, 1),                   # 16-byte copies
    (dict(split=64), {}, 1),
    (dict(split=128 + 16), {}, 1),
    (dict(hq=64 + 1), {}, 1),
    (dict(hq=34), {}, 2),                                     # 17 query heads per KV head
    ({}, dict(D=96), 2),
    ({}, dict(bs=8), 2),
    (dict(max_ctx=-1), {}, 1),
    (dict(softcap=float("nan")), {}, 1),
])
def test_refusals(lib, kw, ckw, code):
    a = dict(hq=32)
    a.update(kw)
    assert chunk(lib, desc(num_blocks=64, **ckw), **a) == code, lib.pkv_last_error()
