"""E2M1 stores on the GPU where a code or a scale can fall on either side: every
border of every scale and its neighbours, every bf16 below a group's largest
value, and the values that are none (NaN, infinities, zeros of both signs),
through every way into a cache."""

import numpy as np
import pytest
import torch

import paged_kv_cache_222_gb300 as pkv
from oracle import formats as F

from . import e2m1_exact as Q
from . import e2m1_support as E

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda", 0)
f32 = np.float32


def store(x, src, ks=None, way="append", **kw):
    """(codes [n, D], scale codes [n, D / 16]) of K and of V after rows x [n, D] went in as both, one head."""
    n, D = x.shape
    bs = 16
    cache = [torch.full((-(-n // bs), 1, bs, D // 2 + D // 16), 0x5A, dtype=torch.uint8, device=DEV) for _ in range(2)]
    k = torch.from_numpy(x).to(DEV, torch.bfloat16 if src == "bf16" else torch.float32)[:, None].contiguous()
    slots = torch.arange(n, device=DEV).flip(0).contiguous()
    s = None if ks is None else torch.from_numpy(ks).to(DEV)[:, None].contiguous()
    if way == "append":
        pkv.append(k, k, slots, *cache, s, s)
    else:
        rd = kw.pop("rotary_dim")
        pkv.rotary_append(k, k, k, slots, torch.zeros(rd // 2, dtype=torch.float64, device=DEV), slots, *cache, s, s, **kw)
    assert pkv.device_error(DEV) == 0
    return [tuple(a[:, 0][slots.cpu().numpy()] for a in E.token_bytes(c)) for c in cache]


def groups_of(values, first, D):
    """Rows [n, D] whose groups of 16 hold `first` (per row of values) and then the row's values, padded with it."""
    m = values.shape[1]
    per = -(-m // 15)
    g = np.broadcast_to(first[:, None, None], (len(first), per, 16)).astype(f32).copy()
    flat = np.broadcast_to(first[:, None], (len(first), per * 15)).astype(f32).copy()
    flat[:, :m] = values
    g[..., 1:] = flat.reshape(len(first), per, 15)
    g = g.reshape(-1, 16)
    pad = -len(g) % (D // 16)
    return np.concatenate([g, np.repeat(g[:1], pad, 0)]).reshape(-1, D)


def check(x, src, s=None, scale=None):
    """Against the exact decisions (`s`: each group's scale, where it is known beforehand)."""
    for codes, sc in store(x, src, scale):
        y = x if scale is None else F.f32_div(x, scale[:, None])
        g = y.reshape(-1, 16)
        want = Q.exact_scale(np.abs(g).max(-1))
        assert (sc.reshape(-1) == want).all()
        assert s is None or (F.e4m3_to_f64(want) == s).all()
        v = F.e4m3_to_f64(want)[:, None]
        ok = v[:, 0] > 0
        assert (codes.reshape(-1, 16)[ok] == Q.exact_codes(g[ok], v[ok])).all()
        assert not codes.reshape(-1, 16)[~ok].any()


@pytest.mark.parametrize("D", [64, 128])
def test_every_border_of_every_scale(D):
    x, _ = Q.near_borders()
    rows = groups_of(x, 6.0 * Q.SCALES, D)
    check(rows, "f32", None)
    # the same after a division by the head's scale that is exact, and one that is not
    n = len(rows)
    check(rows * f32(0.25), "f32", scale=np.full(n, 0.25, dtype=f32))
    check(rows * f32(0.3), "f32", scale=np.full(n, 0.3, dtype=f32))


def test_borders_of_the_scales():
    a = Q.around(6.0 * np.unique(np.concatenate([Q.E4M3[1:], (Q.E4M3[1:] + Q.E4M3[:-1]) / 2])), range(-8, 9)).ravel()
    rng = np.random.default_rng(3)
    g = (rng.uniform(-1, 1, (len(a), 16)) * a[:, None]).astype(f32)
    g[np.arange(len(a)), rng.integers(0, 16, len(a))] = a * rng.choice([-1, 1], len(a)).astype(f32)
    g = np.concatenate([g, np.ones((-len(g) % 8, 16), dtype=f32)])
    check(g.reshape(-1, 128), "f32")


@pytest.mark.parametrize("src", ["bf16", "f32"])
def test_groups_past_the_largest_scale(src):
    # scale 448 whatever the largest value: quotients from 6 on saturate; from 8 on they are divided
    top = np.array([2784.0, 3328.0, 3584.0, 3600.0, 1e4, 1e20, 3e38], dtype=f32)
    top = torch.from_numpy(top).bfloat16().float().numpy() if src == "bf16" else top
    x = Q.around(448.0 * Q.BORDERS, range(-20, 21)).reshape(1, -1)
    if src == "bf16":
        x = np.unique(torch.from_numpy(x).bfloat16().float().numpy())[None]
    x = np.concatenate([x, -x, np.array([[2500.0, 2688.0, 3100.5, 3500.0]], dtype=f32)], axis=1)
    x = torch.from_numpy(x).bfloat16().float().numpy() if src == "bf16" else x
    check(groups_of(np.repeat(x, len(top), 0).clip(-top[:, None], top[:, None]), top, 64), src)


@pytest.mark.parametrize("D", [64, 128])
def test_every_bf16_below_a_groups_largest(D):
    # of every scale: the largest bf16 whose group gets it, and every bf16 from 2^-8 of the scale up to that
    bits = np.arange(1, 0x7F80, dtype=np.int32) << 16
    every = bits.view(f32)
    code = Q.exact_scale(every)
    rows = []
    for c in range(1, 0x7F):
        mine = every[code == c]
        top = mine.max() if c < 0x7E else f32(3584.0)                  # (the last scale's: up to what is not divided)
        v = every[(every <= top) & (every >= F.e4m3_to_f64(np.uint8(c)) * 2.0 ** -8)]
        v = v * np.where(np.arange(v.size) % 2, -1, 1).astype(f32)
        rows.append(groups_of(v[None], np.array([top]), D))
    check(np.concatenate(rows), "bf16")


def specials(D, src):
    x = E.special_rows(D)
    if src == "bf16":
        x = torch.from_numpy(x).bfloat16().float().numpy()
        assert np.isnan(x).any() and np.isinf(x).any()
    return x


def head_scales(n):
    return np.array([0.125, 0.37, 3.0, 1e-3, 64.0, 1.0], dtype=f32)[np.arange(n) % 6]


@pytest.mark.parametrize("src", ["bf16", "f32"])
@pytest.mark.parametrize("scaled", [False, True])
@pytest.mark.parametrize("D", [64, 128])
def test_values_that_are_none_through_append(D, scaled, src):
    x = specials(D, src)
    ks = head_scales(len(x)) if scaled else None
    with np.errstate(over="ignore"):
        want = F.e2m1_rows(x, ks)
    for got in store(x, src, ks):
        assert (got[0] == want[0]).all() and (got[1] == want[1]).all()


@pytest.mark.parametrize("src", ["bf16", "f32"])
@pytest.mark.parametrize("scaled", [False, True])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("D,rd", [(64, 64), (64, 16), (64, 48), (128, 128), (128, 64), (128, 80)])
def test_values_that_are_none_through_rotary_append(D, rd, interleaved, scaled, src):
    x = specials(D, src)
    ks = head_scales(len(x)) if scaled else None
    # an angle of zero, as the formula has it in binary32: infinity times its sine is NaN
    turned = x.copy()
    a, b = (x[:, 0:rd:2], x[:, 1:rd:2]) if interleaved else (x[:, :rd // 2], x[:, rd // 2:rd])
    with np.errstate(invalid="ignore", over="ignore"):
        p, q = a * f32(1) - b * f32(0), b * f32(1) + a * f32(0)
        if interleaved:
            turned[:, 0:rd:2], turned[:, 1:rd:2] = p, q
        else:
            turned[:, :rd // 2], turned[:, rd // 2:rd] = p, q
        wants = F.e2m1_rows(turned, ks), F.e2m1_rows(x, ks)
    for got, want in zip(store(x, src, ks, way="rotary", rotary_dim=rd, interleaved=interleaved), wants):
        assert (got[1] == want[1]).all()
        assert (got[0] == want[0]).all()


def test_what_was_promised_of_them_reads_back():
    # a group that holds a NaN reads as NaN, infinities saturate, a tiny group is zeros
    x = np.ones((4, 64), dtype=f32)
    x[0, 20], x[1, 3], x[2, 40], x[3, 16:32] = np.nan, np.inf, -np.inf, 6 * 2.0 ** -10
    for src in ("bf16", "f32"):
        k = torch.from_numpy(x).to(DEV, torch.bfloat16 if src == "bf16" else torch.float32)[:, None].contiguous()
        cache = [pkv.e2m1_cache(1, 1, 16, 64, device=DEV) for _ in range(2)]
        slots = torch.arange(4, device=DEV)
        pkv.append(k, k, slots, *cache)
        for y in pkv.read_tokens(slots, *cache, dtype=torch.float32):
            y = y[:, 0].cpu().numpy()
            # (ones: a scale of E4M3(1 / 6) = 11 / 64, of which 1 is 5.8, code 6)
            assert np.isnan(y[0, 16:32]).all() and (np.delete(y[0], np.arange(16, 32)) == 6 * 11 / 64).all()
            assert y[1, 3] == 2688 and y[2, 40] == -2688 and not y[3, 16:32].any()
            assert np.isfinite(y[1:]).all()
