"""Host side of E2M1 caches and of rotary positions of several axes: the
format's own pins, what the calls refuse, the helpers (no GPU)."""

import ctypes
import math

import numpy as np
import pytest
import torch

import paged_kv_cache_222_gb300 as pkv
from oracle import formats as F
from paged_kv_cache_222_gb300 import _lib as L
from paged_kv_cache_222_gb300 import build as B

from . import e2m1_support as E

FAKE = 0x10000      # aligned, never dereferenced


@pytest.fixture(scope="module")
def lib():
    B.build()
    return L.load()


def desc(**kw):
    d = dict(num_blocks=64, block_size=16, num_kv_heads=8, head_dim=128, dtype=L.PKV_E2M1)
    d.update(kw)
    return L.CacheDesc(d["num_blocks"], d["block_size"], d["num_kv_heads"], d["head_dim"], d["dtype"])


# ---------------------------------------------------------------- the format

def test_values():
    assert F.E2M1_VALUES[:8].tolist() == [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]
    assert (F.E2M1_VALUES[8:] == -F.E2M1_VALUES[:8]).all() and math.copysign(1, F.E2M1_VALUES[8]) == -1


def test_codes_round_to_nearest_even():
    x = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0, 7.0, np.inf, 0.2500001, 0.7499999, -5.0, -0.0, -0.1],
                 dtype=np.float32)
    assert F.e2m1_encode(x).tolist() == [0, 2, 2, 4, 4, 6, 6, 7, 7, 7, 1, 1, 14, 8, 8]


def test_groups():
    x = np.zeros((1, 32), dtype=np.float32)
    x[0, :3] = [6.0, -1.5, 0.26]                   # scale 1
    x[0, 16] = 6 * 2.0 ** -10                      # its scale is a tie with zero: zeros
    codes, sc = F.e2m1_rows(x)
    assert sc.tolist() == [[0x38, 0]] and codes[0, :3].tolist() == [7, 11, 1] and not codes[0, 16:].any()
    x[0, 20] = np.nan
    codes, sc = F.e2m1_rows(x)
    assert sc[0, 1] == 0x7F and np.isnan(F.e2m1_values(F.e2m1_pack(codes[None, None], sc[None, None]))[0, 0, 0, 16:]).all()
    # a head's scale divides first
    codes2, sc2 = F.e2m1_rows(x[:, :16] * np.float32(0.125), np.array([0.125], dtype=np.float32))
    assert (codes2 == codes[:, :16]).all() and (sc2 == sc[:, :1]).all()


def test_packing_is_undone():
    rng = np.random.default_rng(1)
    codes = rng.integers(0, 16, (3, 2, 16, 64)).astype(np.uint8)
    sc = rng.integers(0, 256, (3, 2, 16, 4)).astype(np.uint8)
    b = F.e2m1_pack(codes, sc)
    assert b.shape == (3, 2, 16, 36)
    c, s = F.e2m1_unpack(b)
    assert (c == codes).all() and (s == sc).all()
    flat = b.reshape(3, 2, -1)
    assert flat[1, 1, 5 * 32 + 7] == codes[1, 1, 5, 14] | codes[1, 1, 5, 15] << 4
    assert flat[1, 1, 16 * 32 + 5 * 4 + 2] == sc[1, 1, 5, 2]


def test_quotients_in_binary32_decide_as_exact_ones_do():
    # a value over its scale rounds to a code's border only if it lies on it, so
    # that the code is the one of the exact quotient
    codes, sc = F.e2m1_rows(E.special_rows(128))
    x = E.special_rows(128).reshape(-1, 16).astype(np.float64)
    s = F.e4m3_to_f64(sc).reshape(-1)
    fine = np.isfinite(x).all(-1) & (s > 0)
    y = np.minimum(np.abs(x[fine]) / s[fine, None], 6.0)
    got = np.abs(F.E2M1_VALUES[codes.reshape(-1, 16)[fine]])
    best = np.abs(y[..., None] - F.E2M1_VALUES[:8]).min(-1)
    assert np.allclose(np.abs(y - got), best, rtol=0, atol=1e-6)


# ---------------------------------------------------------------- refusals

def append(lib, c, **kw):
    a = dict(k=FAKE, v=FAKE, src=L.PKV_BF16, n=4, slots=FAKE, kc=FAKE, vc=FAKE, ks=None, vs=None, stride=0)
    a.update(kw)
    return lib.pkv_append(a["k"], a["v"], a["src"], a["n"], a["slots"], a["kc"], a["vc"], ctypes.byref(c), a["ks"],
                          a["vs"], a["stride"], None)


@pytest.mark.parametrize("kw,dkw,code", [
    (dict(n=-1), {}, 1), (dict(src=L.PKV_E4M3), {}, 1), (dict(src=L.PKV_E2M1), {}, 1), (dict(ks=FAKE), {}, 1),
    (dict(vs=FAKE), {}, 1), (dict(ks=FAKE, vs=FAKE, stride=-1), {}, 1), (dict(ks=FAKE + 2, vs=FAKE), {}, 1),
    (dict(k=FAKE + 8), {}, 1), (dict(kc=FAKE + 8), {}, 1), (dict(slots=None), {}, 1), ({}, dict(head_dim=96), 2),
    ({}, dict(block_size=8), 2), ({}, dict(dtype=4), 1), ({}, dict(dtype=-1), 1),
])
def test_append_refuses(lib, kw, dkw, code):
    assert append(lib, desc(**dkw), **kw) == code, lib.pkv_last_error()


def read(lib, c, **kw):
    a = dict(slots=FAKE, n=4, kc=FAKE, vc=FAKE, ks=None, vs=None, stride=0, ko=FAKE, vo=FAKE, dt=L.PKV_BF16)
    a.update(kw)
    return lib.pkv_read_tokens(a["slots"], a["n"], a["kc"], a["vc"], ctypes.byref(c), a["ks"], a["vs"], a["stride"],
                               a["ko"], a["vo"], a["dt"], None)


@pytest.mark.parametrize("kw,dkw,code", [
    (dict(n=-1), {}, 1), (dict(dt=L.PKV_E4M3), {}, 1), (dict(ks=FAKE), {}, 1), (dict(slots=None), {}, 1),
    (dict(slots=FAKE + 4), {}, 1), (dict(ko=FAKE + 8), {}, 1), (dict(vo=None), {}, 1), (dict(kc=None), {}, 1),
    ({}, dict(dtype=L.PKV_E4M3), 1), (dict(ks=FAKE, vs=FAKE), dict(dtype=L.PKV_BF16), 1), ({}, dict(head_dim=32), 2),
])
def test_read_refuses(lib, kw, dkw, code):
    assert read(lib, desc(**dkw), **kw) == code, lib.pkv_last_error()


def test_empty_calls_are_noops(lib):
    assert append(lib, desc(), n=0, k=None, v=None, slots=None, kc=None, vc=None) == 0
    assert read(lib, desc(), n=0, slots=None, ko=None, vo=None) == 0


def test_the_other_attentions_refuse_e2m1(lib):
    c, plan = desc(), L.DecodePlan()
    assert lib.pkv_decode_plan(1, 64, ctypes.byref(c), 100, 0, 0, ctypes.byref(plan)) == 2
    assert lib.pkv_cascade_plan(1, 64, ctypes.byref(c), 16, 100, 0, ctypes.byref(plan)) == 2
    assert lib.pkv_multi_query_plan(1, 2, 64, ctypes.byref(c), 100, 0, 0, ctypes.byref(plan)) == 2
    assert b"pkv_chunk_attention" in lib.pkv_last_error()
    assert lib.pkv_decode_attention_ex(FAKE, 1, 64, FAKE, FAKE, ctypes.byref(c), FAKE, 8, FAKE, 100, 0.1, FAKE, None,
                                       None, 0, None, 0, 0, None) == 2
    assert lib.pkv_decode_attention_append(FAKE, 1, 64, FAKE, FAKE, ctypes.byref(c), FAKE, FAKE, 0, FAKE, 8, FAKE, 100,
                                           0.1, FAKE, None, None, 0, None, 0, 0, None) == 2


def axes_call(lib, c, **kw):
    a = dict(n=4, hq=64, pos=FAKE, ps=4, na=3, axes=FAKE, f=FAKE, rd=128)
    a.update(kw)
    return lib.pkv_rotary_append_axes(FAKE, 64 * 128, FAKE, 8 * 128, FAKE, 8 * 128, L.PKV_BF16, a["n"], a["hq"], a["pos"],
                                      a["ps"], a["na"], a["axes"], a["f"], a["rd"], 0, 1.0, FAKE, FAKE, FAKE,
                                      ctypes.byref(c), None, None, 0, FAKE + 65536, 64 * 128, None)


@pytest.mark.parametrize("kw", [dict(na=0), dict(na=-1), dict(na=65536), dict(ps=-1), dict(axes=None),
                                dict(axes=FAKE + 2), dict(pos=None), dict(pos=FAKE + 4)])
def test_rotary_axes_refuse(lib, kw):
    assert axes_call(lib, desc(), **kw) == 1, lib.pkv_last_error()


def test_rotary_axes_of_no_tokens(lib):
    assert axes_call(lib, desc(), n=0, axes=None) == 0


# ---------------------------------------------------------------- helpers

def test_rotary_axes():
    assert pkv.rotary_axes((2, 1, 3)).tolist() == [0, 0, 1, 2, 2, 2]
    assert pkv.rotary_axes((2, 1, 3), mixed=True).tolist() == [0, 1, 2, 0, 2, 2]
    assert pkv.rotary_axes((4,)).tolist() == [0] * 4 and pkv.rotary_axes((0, 2)).tolist() == [1, 1]
    assert pkv.rotary_axes((16, 24, 24)).dtype == torch.int32
    for bad in ((), (0, 0), (3, -1)):
        with pytest.raises(ValueError):
            pkv.rotary_axes(bad)


def test_cache_tensors():
    c = pkv.e2m1_cache(5, 3, 16, 128, device="cpu")
    assert c.shape == (5, 3, 16, 72) and c.dtype == torch.uint8 and not c.any()
    d = pkv.cache_desc(c)
    assert (d.num_blocks, d.num_kv_heads, d.block_size, d.head_dim, d.dtype) == (5, 3, 16, 128, pkv.PKV_E2M1)
    d = pkv.cache_desc(pkv.e2m1_cache(2, 1, 32, 64, device="cpu"))
    assert (d.head_dim, d.dtype) == (64, pkv.PKV_E2M1)
    assert pkv.cache_desc(torch.zeros((2, 1, 16, 64), dtype=torch.uint8)).dtype == pkv.PKV_E4M3
    with pytest.raises(ValueError):
        pkv.e2m1_cache(5, 3, 16, 72, device="cpu")


def test_python_checks_come_before_the_library():
    c = pkv.e2m1_cache(5, 3, 16, 128, device="cpu")
    k = torch.zeros((2, 3, 128))
    with pytest.raises(ValueError):
        pkv.append(k, k, torch.zeros(2, dtype=torch.int64), c, c)       # caches not on a GPU
    with pytest.raises(ValueError):
        pkv.read_tokens(torch.zeros(2, dtype=torch.int64), c, c)
    with pytest.raises(TypeError):
        pkv.read_tokens(torch.zeros(2, dtype=torch.int64), c, c, dtype=torch.float16)
