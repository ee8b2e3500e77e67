"""Host side of extend_tables and truncate_tables: refusals, and the oracle's
own pins against the host block manager (no GPU)."""

import ctypes

import numpy as np
import pytest
import torch

import paged_kv_cache_222_gb300 as pkv
from oracle import tables as OT
from paged_kv_cache_222_gb300 import _lib as L
from paged_kv_cache_222_gb300 import build as B

FAKE = 0x10000      # aligned, never dereferenced


@pytest.fixture(scope="module")
def lib():
    B.build()
    return L.load()


def desc(**kw):
    d = dict(num_blocks=64, block_size=16, num_kv_heads=8, head_dim=128, dtype=L.PKV_E2M1)
    d.update(kw)
    return L.CacheDesc(d["num_blocks"], d["block_size"], d["num_kv_heads"], d["head_dim"], d["dtype"])


def extend(lib, c, **kw):
    a = dict(t=FAKE, mb=8, B=3, past=FAKE, new=FAKE, fb=FAKE, cap=10, fc=FAKE, most=16, ctx=FAKE, qs=FAKE, bst=FAKE,
             slots=FAKE, pos=FAKE, fo=FAKE, lack=FAKE, out=True)
    a.update(kw)
    step = L.TableStep(a["ctx"], a["qs"], a["bst"], a["slots"], a["pos"], a["fo"], a["lack"])
    return lib.pkv_extend_tables(a["t"], a["mb"], a["B"], a["past"], a["new"], a["fb"], a["cap"], a["fc"],
                                 ctypes.byref(c), a["most"], ctypes.byref(step) if a["out"] else None, None)


@pytest.mark.parametrize("kw,dkw,code", [
    (dict(B=-1), {}, 1), (dict(B=65536), {}, 1), (dict(mb=0), {}, 1), (dict(mb=1 << 28), {}, 1), (dict(cap=-1), {}, 1),
    (dict(most=-1), {}, 1), (dict(most=1 << 31), {}, 1), (dict(t=None), {}, 1), (dict(past=None), {}, 1),
    (dict(new=None), {}, 1), (dict(fb=None), {}, 1), (dict(fc=None), {}, 1), (dict(ctx=None), {}, 1),
    (dict(qs=None), {}, 1), (dict(bst=None), {}, 1), (dict(slots=None), {}, 1), (dict(pos=None), {}, 1),
    (dict(fo=None), {}, 1), (dict(lack=None), {}, 1), (dict(out=False), {}, 1), (dict(slots=FAKE + 4), {}, 1),
    (dict(pos=FAKE + 4), {}, 1), (dict(qs=FAKE + 2), {}, 1), (dict(t=FAKE + 1), {}, 1), ({}, dict(block_size=8), 2),
    ({}, dict(num_blocks=0), 1), ({}, dict(dtype=7), 1),
])
def test_extend_refuses(lib, kw, dkw, code):
    assert extend(lib, desc(**dkw), **kw) == code, lib.pkv_last_error()


def truncate(lib, c, **kw):
    a = dict(t=FAKE, mb=8, B=3, ctx=FAKE, keep=FAKE, fb=FAKE, cap=10, fc=FAKE, bst=FAKE, fo=FAKE)
    a.update(kw)
    return lib.pkv_truncate_tables(a["t"], a["mb"], a["B"], a["ctx"], a["keep"], a["fb"], a["cap"], a["fc"],
                                   ctypes.byref(c), a["bst"], a["fo"], None)


@pytest.mark.parametrize("kw", [dict(B=-1), dict(B=65536), dict(mb=0), dict(cap=-1), dict(t=None), dict(ctx=None),
                                dict(keep=None), dict(fb=None), dict(fc=None), dict(bst=None), dict(fo=None),
                                dict(fo=FAKE + 2), dict(keep=FAKE + 1)])
def test_truncate_refuses(lib, kw):
    assert truncate(lib, desc(), **kw) == 1, lib.pkv_last_error()


def test_python_checks_come_before_the_library():
    cache = torch.zeros((4, 2, 16, 64), dtype=torch.bfloat16)
    i = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError):
        pkv.extend_tables(torch.zeros((2, 4), dtype=torch.int32), i, i, i, i[:1], cache, 8)
    with pytest.raises(ValueError):
        pkv.truncate_tables(torch.zeros((2, 4), dtype=torch.int32), i, i, i, i[:1], cache)


def test_the_model_takes_blocks_as_the_host_manager_does(lib):
    # same stack, same order: tables and slots agree step by step
    bs, nb = 16, 40
    bm = pkv.BlockManager(nb, bs)
    for s in range(3):
        bm.add_sequence(s)
    free, count = np.arange(nb, dtype=np.int32), nb
    table, past = np.full((3, 20), -1, dtype=np.int32), np.zeros(3, dtype=np.int32)
    rng = np.random.default_rng(1)
    for _ in range(12):
        new = rng.integers(0, 20, 3).astype(np.int32)
        slots, _ = bm.append([0, 1, 2], new)
        table, past, qs, sl, pos, _, count, lacking, good = OT.extend(table, past, new, free, count, bs, 64, nb)
        assert good and lacking == 0 and count == bm.num_free()
        assert (sl[:qs[-1]] == slots).all() and (sl[qs[-1]:] == -1).all()
        want, lens = bm.block_tables([0, 1, 2], 20)
        assert (lens == past).all() and ((want == table) | (want == -1)).all()


def test_the_model_undoes_what_it_did():
    rng = np.random.default_rng(2)
    nb, bs = 60, 16
    free = rng.permutation(nb).astype(np.int32)
    past, new = np.array([0, 5, 16, 31]), np.array([40, 0, 1, 100])
    table = np.full((4, 10), -1, dtype=np.int32)
    for b, p in enumerate(past):
        for j in range(-(-p // bs)):
            table[b, j] = nb + 10 * b + j             # ids that are none of the stack's
    t, ctx, *_, block_starts, count, lacking, good = OT.extend(table, past, new, free, 50, bs, 200, 200)
    assert good and lacking == 0 and count == 50 - block_starts[-1]
    back, n, good = OT.truncate(t, ctx, past, free, count, bs, 200)
    assert good and n == 50 and (back == free).all()
    # too few: nothing
    t, ctx, qs, sl, _, _, n, lacking, good = OT.extend(table, past, new, free, 3, bs, 200, 200)
    assert n == 3 and lacking == block_starts[-1] - 3 and (sl == -1).all() and not qs.any() and (ctx == past).all()
