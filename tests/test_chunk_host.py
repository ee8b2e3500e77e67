"""Host side of the chunk, rotary and compaction calls: refusals, plans, the
frequency tables, truncation and the oracle's own pins (no GPU)."""

import ctypes
import math

import numpy as np
import pytest
import torch

import paged_kv_cache_222_gb300 as pkv
from oracle import chunk as OC
from paged_kv_cache_222_gb300 import _lib as L
from paged_kv_cache_222_gb300 import build as B

FAKE = 0x10000      # aligned, never dereferenced


@pytest.fixture(scope="module")
def lib():
    B.build()
    return L.load()


def desc(**kw):
    d = dict(num_blocks=64, block_size=16, num_kv_heads=8, head_dim=128, dtype=L.PKV_BF16)
    d.update(kw)
    return L.CacheDesc(d["num_blocks"], d["block_size"], d["num_kv_heads"], d["head_dim"], d["dtype"])


def chunk(lib, c, **kw):
    a = dict(q=FAKE, T=10, qs=FAKE, batch=2, mq=8, hq=64, kc=FAKE, vc=FAKE, bt=FAKE, mb=8, cl=FAKE, max_ctx=100,
             scale=0.125, softcap=0.0, window=0, slopes=None, prefix=None, out=FAKE, ks=None, vs=None, stride=0,
             ws=None, ws_bytes=0, split=0)
    a.update(kw)
    m = L.ScoreMods(a["softcap"], a["window"], a["slopes"], a["prefix"])
    return lib.pkv_chunk_attention(a["q"], a["T"], a["qs"], a["batch"], a["mq"], a["hq"], a["kc"], a["vc"],
                                   ctypes.byref(c), a["bt"], a["mb"], a["cl"], a["max_ctx"], a["scale"],
                                   ctypes.byref(m), a["out"], a["ks"], a["vs"], a["stride"], a["ws"], a["ws_bytes"],
                                   a["split"], None)


@pytest.mark.parametrize("kw,dkw,code", [
    (dict(T=-1), {}, 1), (dict(batch=-1), {}, 1), (dict(batch=65536), {}, 1), (dict(mq=0), {}, 1),
    (dict(hq=60), {}, 1), (dict(hq=8 * 17), {}, 2), (dict(max_ctx=-1), {}, 1), (dict(max_ctx=129), {}, 1),
    (dict(mb=0), {}, 1), (dict(scale=0.0), {}, 1), (dict(scale=-1.0), {}, 1), (dict(scale=math.nan), {}, 1),
    (dict(scale=math.inf), {}, 1), (dict(softcap=-1.0), {}, 1), (dict(softcap=math.inf), {}, 1),
    (dict(softcap=math.nan), {}, 1), (dict(softcap=1e-45), {}, 1), (dict(softcap=3e38), {}, 1), (dict(window=-1), {}, 1), (dict(q=None), {}, 1), (dict(qs=None), {}, 1),
    (dict(out=FAKE + 4), {}, 1), (dict(q=FAKE + 2), {}, 1), (dict(kc=FAKE + 8), {}, 1), (dict(qs=FAKE + 2), {}, 1),
    (dict(slopes=FAKE + 1), {}, 1), (dict(prefix=FAKE + 1), {}, 1), (dict(ks=FAKE, vs=FAKE), {}, 1),
    ({}, dict(dtype=L.PKV_E4M3), 1), ({}, dict(dtype=L.PKV_F32), 1), ({}, dict(head_dim=96), 2),
    ({}, dict(block_size=8), 2), ({}, dict(num_blocks=0), 1), (dict(split=64), {}, 1), (dict(split=-128), {}, 1),
    (dict(split=128 * 200), {}, 1), (dict(stride=-1, ks=FAKE, vs=FAKE), dict(dtype=L.PKV_E4M3), 1),
])
def test_chunk_refuses_on_the_host(lib, kw, dkw, code):
    assert chunk(lib, desc(**dkw), **kw) == code, lib.pkv_last_error()
    assert lib.pkv_last_error()


def test_empty_chunk_calls_are_noops(lib):
    assert chunk(lib, desc(), batch=0, T=0, q=None, out=None, qs=None) == 0
    assert chunk(lib, desc(), T=0, q=None, out=None, qs=None) == 0


def rotary(lib, c, **kw):
    a = dict(q=FAKE, qs=64 * 128, k=FAKE, ks=8 * 128, v=FAKE, vs=8 * 128, src=L.PKV_BF16, n=4, hq=64, pos=FAKE,
             f=FAKE, rd=128, inter=0, mag=1.0, slots=FAKE, kc=FAKE, vc=FAKE, ksc=None, vsc=None, stride=0,
             out=FAKE + 65536, os=64 * 128)
    a.update(kw)
    return lib.pkv_rotary_append(a["q"], a["qs"], a["k"], a["ks"], a["v"], a["vs"], a["src"], a["n"], a["hq"],
                                 a["pos"], a["f"], a["rd"], a["inter"], a["mag"], a["slots"], a["kc"], a["vc"],
                                 ctypes.byref(c), a["ksc"], a["vsc"], a["stride"], a["out"], a["os"], None)


@pytest.mark.parametrize("kw,dkw,code", [
    (dict(n=-1), {}, 1), (dict(src=L.PKV_E4M3), {}, 1), (dict(hq=0), {}, 1), (dict(rd=8), {}, 2), (dict(rd=24), {}, 2),
    (dict(rd=144), {}, 2), (dict(rd=0), {}, 2), (dict(inter=2), {}, 1), (dict(mag=math.nan), {}, 1),
    (dict(qs=64 * 128 - 8), {}, 1), (dict(ks=8), {}, 1), (dict(vs=8 * 128 + 4), {}, 1), (dict(os=0), {}, 1),
    (dict(q=None), {}, 1), (dict(pos=None), {}, 1), (dict(f=None), {}, 1), (dict(slots=None), {}, 1),
    (dict(k=FAKE + 8), {}, 1), (dict(out=FAKE + 8), {}, 1), (dict(pos=FAKE + 4), {}, 1), (dict(f=FAKE + 4), {}, 1),
    (dict(out=FAKE, src=L.PKV_F32, os=64 * 128), {}, 1), (dict(out=FAKE, os=65 * 128), {}, 1),
    (dict(ksc=FAKE, vsc=FAKE), {}, 1), ({}, dict(dtype=L.PKV_E4M3), 1), ({}, dict(head_dim=96), 2),
])
def test_rotary_refuses_on_the_host(lib, kw, dkw, code):
    assert rotary(lib, desc(**dkw), **kw) == code, lib.pkv_last_error()


def test_empty_rotary_call_is_a_noop(lib):
    assert rotary(lib, desc(), n=0, q=None, k=None, v=None, out=None) == 0


def compact(lib, c, **kw):
    a = dict(kc=FAKE, vc=FAKE, bt=FAKE, mb=8, batch=2, keep=FAKE, n=10, ks=FAKE, dst=None, mk=10)
    a.update(kw)
    return lib.pkv_compact_tokens(a["kc"], a["vc"], ctypes.byref(c), a["bt"], a["mb"], a["batch"], a["keep"], a["n"],
                                  a["ks"], a["dst"], a["mk"], None)


@pytest.mark.parametrize("kw,dkw,code", [
    (dict(batch=-1), {}, 1), (dict(n=-1), {}, 1), (dict(mk=-1), {}, 1), (dict(mb=0), {}, 1), (dict(keep=None), {}, 1),
    (dict(ks=None), {}, 1), (dict(bt=None), {}, 1), (dict(kc=FAKE + 8), {}, 1), (dict(dst=FAKE + 2), {}, 1),
    ({}, dict(head_dim=96), 2), ({}, dict(num_kv_heads=9000), 2),
])
def test_compact_refuses_on_the_host(lib, kw, dkw, code):
    assert compact(lib, desc(**dkw), **kw) == code, lib.pkv_last_error()


def test_empty_compact_calls_are_noops(lib):
    assert compact(lib, desc(), batch=0) == 0
    assert compact(lib, desc(), n=0, keep=None) == 0


def test_chunk_plans(lib):
    c = desc(num_blocks=1 << 20)
    p = pkv.chunk_plan(8192, 2, 4096, 64, c, 8192)
    assert (p.mode, p.max_splits, p.workspace_bytes) == (4, 1, 0)
    p = pkv.chunk_plan(1, 1, 1, 64, c, 131072)               # one decode: split
    assert p.workers == 1 and p.max_splits > 1
    n = 64 * p.max_splits
    assert p.workspace_bytes >= n * 130 * 4
    # a window without prefixes bounds what is split
    w = pkv.chunk_plan(1, 1, 1, 64, c, 131072, window=1024)
    assert w.max_splits < p.max_splits
    assert pkv.chunk_plan(1, 1, 1, 64, c, 131072, window=1024, has_prefix=True).max_splits == p.max_splits
    with pytest.raises(pkv.PkvError):
        pkv.chunk_plan(1, 1, 1, 60, c, 100)


@pytest.mark.parametrize("dkw", [{}, dict(head_dim=64), dict(dtype=pkv.PKV_E4M3), dict(head_dim=64, dtype=pkv.PKV_E4M3)])
@pytest.mark.parametrize("group", [1, 8, 16])
def test_plans_of_single_tokens(lib, dkw, group):
    # every size: the pieces hold the context, fit the block list and are whole
    # steps; nothing to do is a plan too
    c = desc(num_blocks=1 << 20, **dkw)
    h = c.num_kv_heads
    assert pkv.chunk_plan(0, 0, 1, group * h, c, 0).workspace_bytes == 0
    for batch in (1, 2, 3, 8, 17, 64, 300, 4000):
        for ctx in (1, 64, 100, 1000, 1025, 2048, 2049, 8192, 30000, 200001, 1 << 21):
            p = pkv.chunk_plan(batch, batch, 1, group * h, c, ctx)
            assert p.workers == 1 and p.split_tokens % 64 == 0
            assert 64 <= p.split_tokens <= 1024 * c.block_size
            steps = -(-ctx // 64) * 64
            assert (p.max_splits - 1) * p.split_tokens < steps <= p.max_splits * p.split_tokens


@pytest.mark.parametrize("dkw", [{}, dict(head_dim=64), dict(dtype=pkv.PKV_E4M3), dict(block_size=32)])
@pytest.mark.parametrize("T,B,mq", [(200_000, 2, 100_000), (8192, 2, 4096), (1 << 20, 64, 1 << 20), (40, 1, 40)])
def test_plans_at_the_longest_contexts(lib, T, B, mq, dkw):
    # sizes of the tcgen05 kernel's splits stay 32-bit numbers up to the last
    # bound there is; contexts count up to 2^31 - 256
    c = desc(num_blocks=1 << 27, **dkw)
    for ctx in (2 ** 31 - 1, 2 ** 31 - 64, 2 ** 31 - 127, 2 ** 31 - 128, 2 ** 31 - 256, 2 ** 31 - 257, 2 ** 30 + 1):
        for window in (0, 1000, 2 ** 31 - 1):
            p = pkv.chunk_plan(T, B, mq, 64, c, ctx, window=window, has_prefix=window == 1000)
            assert p.workers == 0 and p.split_tokens > 0 and p.split_tokens % 128 == 0 and p.max_splits >= 1
            assert p.split_tokens * p.max_splits >= min(ctx, 2 ** 31 - 256)
            if p.max_splits > 1:
                assert p.workspace_bytes >= T * 64 * p.max_splits * (c.head_dim + 2) * 4


def test_python_checks_come_before_the_library():
    q = torch.zeros((2, 8, 128), dtype=torch.bfloat16)
    kc = torch.zeros((4, 2, 16, 128), dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        pkv.chunk_attention(q, kc, kc, None, None, None, 0.1)       # caches not on a GPU
    with pytest.raises(ValueError):
        pkv.rotary_append(q, q, q, None, None, None, kc, kc)
    with pytest.raises(ValueError):
        pkv.compact_tokens(kc, kc, None, None, None)


def test_rotary_frequencies():
    f = pkv.rotary_frequencies(128)
    assert f.dtype == torch.float64 and f.shape == (64,)
    assert f[0] == 1.0 and abs(f[32].item() - 0.01) < 1e-15
    assert torch.equal(pkv.rotary_frequencies(128, scaling="linear", factor=4.0), f / 4)
    ntk = pkv.rotary_frequencies(128, scaling="ntk", factor=4.0)
    assert ntk[0] == 1.0 and abs(ntk[-1] / f[-1] - 0.25) < 1e-12
    bp = pkv.rotary_frequencies(128, scaling="by_parts", factor=8.0, original_len=8192)
    turns = 8192 * f / (2 * math.pi)
    assert torch.equal(bp[turns >= 32], f[turns >= 32])
    assert torch.allclose(bp[turns <= 1], f[turns <= 1] / 8, rtol=1e-15)
    assert (bp[1:] < bp[:-1]).all()
    for kw in (dict(scaling="other"), dict(scaling="by_parts"), dict(factor=0.0), dict(base=-1.0)):
        with pytest.raises(ValueError):
            pkv.rotary_frequencies(64, **kw)
    with pytest.raises(ValueError):
        pkv.rotary_frequencies(63)


def test_truncate(lib):
    bm = pkv.BlockManager(10, 16)
    bm.add_sequence(1)
    bm.append([1], [100])                       # 7 blocks
    assert bm.num_free() == 3
    bm.truncate(1, 100)
    assert bm.num_free() == 3
    bm.truncate(1, 65)                          # 5 blocks
    assert bm.num_free() == 5 and bm.seq_len(1) == 65
    bm.fork(1, 2)
    bm.truncate(2, 17)                          # shared blocks stay with the parent
    assert bm.num_free() == 5 and bm.seq_len(2) == 17
    first = bm.block_tables([1], 7)[0][0]
    assert bm.ref_count(first[0]) == 2 and bm.ref_count(first[2]) == 1
    slots, cow = bm.append([2], [1])            # its last block is shared: copied first
    assert cow.shape == (1, 2) and cow[0, 0] == first[1]
    bm.truncate(1, 0)
    assert bm.seq_len(1) == 0 and len(bm.table_entries(1)[0]) == 0
    assert bm.ref_count(first[0]) == 1
    slots, _ = bm.append([1], [3])
    assert len(slots) == 3
    for bad in (-1, 4):
        with pytest.raises(pkv.PkvError):
            bm.truncate(1, bad)
    with pytest.raises(pkv.PkvError):
        bm.truncate(9, 0)
    bm.free_sequence(1)
    bm.free_sequence(2)
    assert bm.num_free() == 10


def test_truncate_returns_host_blocks(lib):
    bm = pkv.BlockManager(8, 16)
    bm.set_host_blocks(8)
    bm.add_sequence(5)
    bm.append([5], [64])
    bm.evict(5, [2, 3])
    assert bm.num_free_host() == 6 and bm.host_entries(5) == 2
    bm.truncate(5, 33)
    assert bm.num_free_host() == 7 and bm.host_entries(5) == 1
    bm.stage(5, [2])
    assert bm.host_entries(5) == 0


def test_oracle_visibility():
    assert OC.visible(4, 2).astype(int).tolist() == [[1, 1, 1, 0], [1, 1, 1, 1]]
    assert OC.visible(4, 2, window=2).astype(int).tolist() == [[0, 1, 1, 0], [0, 0, 1, 1]]
    assert OC.visible(4, 2, window=1, prefix=1).astype(int).tolist() == [[1, 0, 1, 0], [1, 0, 0, 1]]
    assert OC.visible(4, 4, prefix=3).astype(int).tolist() == [[1, 1, 1, 0]] * 3 + [[1, 1, 1, 1]]
    assert OC.visible(2, 3).astype(int).tolist() == [[0, 0], [1, 0], [1, 1]]
    assert OC.visible(2, 3, prefix=2)[0].tolist() == [False, False]


def test_oracle_rotation_is_a_rotation():
    x = np.random.default_rng(0).standard_normal((3, 2, 8))
    y = OC.rotate(x, [0, 1, 7], [1.0, 0.1], interleaved=True)
    assert np.allclose(y[0], x[0]) and np.allclose(y[..., 4:], x[..., 4:])
    assert np.allclose(np.hypot(y[..., 0], y[..., 1]), np.hypot(x[..., 0], x[..., 1]))
    z = OC.rotate(x, [0, 1, 7], [1.0, 0.1])
    assert np.allclose(z[1, :, 0], x[1, :, 0] * math.cos(1) - x[1, :, 2] * math.sin(1))
    assert np.allclose(z[1, :, 3], x[1, :, 3] * math.cos(.1) + x[1, :, 1] * math.sin(.1))
