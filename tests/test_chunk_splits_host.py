"""The plan's splits against the kernels' own count of them: a row tile's
visible keys, in tiles of 64 or 128, never make more pieces than the plan has
room for (the merge indexes the workspace by them).  No GPU."""

import numpy as np
import pytest

import paged_kv_cache_222_gb300 as pkv
from paged_kv_cache_222_gb300 import _lib as L
from paged_kv_cache_222_gb300 import build as B


@pytest.fixture(scope="module", autouse=True)
def _built():
    B.build()


def pieces(n, ctx, tile_q, window, prefix, nk, split_tokens):
    """The most pieces of a row tile of a sequence, as the kernels count them
    (and that the pieces cover the tiles)."""
    most = 0
    prefix = min(max(prefix, 0), ctx)
    for i0 in range(0, n, tile_q):
        i1 = min(n, i0 + tile_q) - 1
        pos0, pos1 = ctx - n + i0, ctx - n + i1
        hi = 0 if pos1 < 0 else pos1 + 1
        pre = 0 if pos1 < 0 else prefix
        lo = pos0 - window + 1 if window > 0 and pos0 >= window else 0
        na = -(-pre // nk)
        b0 = max(lo // nk, na)
        tiles = na + max(-(-hi // nk) - b0, 0)
        per = split_tokens // nk
        nsplit = -(-tiles // per) if tiles > per else 1
        each = -(-tiles // nsplit)
        assert each <= per and sum(max(min(each, tiles - s * each), 0) for s in range(nsplit)) == tiles
        most = max(most, nsplit)
    return most


@pytest.mark.parametrize("fp8,D", [(False, 128), (False, 64), (True, 128), (True, 64)])
@pytest.mark.parametrize("group", [1, 3, 7, 8, 16])
def test_pieces_fit_the_plan(fp8, D, group):
    desc = L.CacheDesc(1 << 20, 16, 2, D, pkv.PKV_E4M3 if fp8 else pkv.PKV_BF16)
    rng = np.random.default_rng(group * 1000 + D + fp8)
    checked = 0
    for _ in range(150):
        max_q = int(rng.choice([1, 2, 5, 16, 17, 33, 100, 257, 700, 2000]))
        max_ctx = int(rng.choice([1, 63, 64, 65, 127, 128, 129, 500, 1024, 3001, 9000, 40000]))
        window = int(rng.choice([0, 0, 1, 50, 63, 64, 65, 127, 128, 129, 300, 1024, 5000]))
        has_prefix = bool(rng.random() < 0.4)
        split = int(rng.choice([0, 0, 128, 256, 640, 1024]))
        batch = int(rng.choice([1, 2, 7, 40]))
        T = int(rng.integers(max_q, max_q * batch + 1))
        p = pkv.chunk_plan(T, batch, max_q, 2 * group, desc, max_ctx, window=window, has_prefix=has_prefix,
                           split_tokens=split)
        small = p.workers == 1
        assert small == (max_q * group <= 16)
        tile_q = (16 if small else 256) // group
        assert p.split_tokens % 64 == 0 and (small or p.split_tokens % 128 == 0)
        for _ in range(12):
            n = int(rng.integers(1, max_q + 1))
            ctx = int(rng.integers(0, max_ctx + 1)) if rng.random() < 0.8 else max_ctx
            prefix = int(rng.integers(0, max_ctx + 1)) if has_prefix else 0
            for nk in ((64,) if small else (64, 128)):
                assert pieces(n, ctx, tile_q, window, prefix, nk, p.split_tokens) <= p.max_splits
                checked += 1
    assert checked > 1000


@pytest.mark.parametrize("nk", [64, 128])
def test_every_alignment_of_a_window(nk):
    # the tightest bound: as many queries as a tile has, at each offset
    desc = L.CacheDesc(1 << 20, 16, 1, 128, pkv.PKV_BF16)
    for group, window in [(16, 1), (16, 65), (8, 127), (4, 128), (2, 129), (1, 100)]:
        tile_q = 256 // group
        for split in (128, 256):
            p = pkv.chunk_plan(tile_q, 1, tile_q, group, desc, 3000, window=window, split_tokens=split)
            assert p.workers == 0
            assert all(pieces(tile_q, ctx, tile_q, window, 0, nk, split) <= p.max_splits
                       for ctx in range(2000, 2000 + 2 * nk))
