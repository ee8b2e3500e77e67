"""GPU parity of rotary_append against the float64 oracle, and bit parity of
its append against pkv.append."""

import numpy as np
import pytest
import torch

import paged_kv_cache_222_gb300 as pkv
from oracle import chunk as OC

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda", 0)


def make(n, H_q, H_kv, D, bs, kv, src, far=1 << 20, seed=1, pad=0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    dt = torch.bfloat16 if src == "bf16" else torch.float32
    q, k, v = (torch.randn((n, h, D), generator=g, device=DEV).to(dt) for h in (H_q, H_kv, H_kv))
    nb = -(-max(n, 1) // bs) + 2
    cd = torch.bfloat16 if kv == "bf16" else torch.uint8
    kc = torch.full((nb, H_kv, bs, D), 7, device=DEV, dtype=cd)
    vc = kc.clone()
    pos = torch.randint(-far, far, (n,), generator=g, device=DEV)
    slots = torch.randperm(nb * bs, generator=g, device=DEV)[:n]
    if pad:
        slots[-pad:] = -1
    ks = vs = None
    if kv == "e4m3":
        ks, vs = ((0.5 + torch.rand((n, H_kv), generator=g, device=DEV)) / 64 for _ in range(2))
    return q, k, v, pos, slots, kc, vc, ks, vs


def rows_of(cache, slots):
    bs = cache.shape[2]
    return cache[slots // bs, :, slots % bs]


@pytest.mark.parametrize("n", [1, 5, 700])
@pytest.mark.parametrize("kv,src", [("bf16", "bf16"), ("bf16", "f32"), ("e4m3", "bf16"), ("e4m3", "f32")])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("H_q,H_kv,D,rd,bs", [(8, 2, 128, 128, 16), (5, 1, 64, 64, 32), (3, 3, 128, 64, 16),
                                              (4, 4, 64, 16, 16), (64, 8, 128, 48, 32)])
def test_matches_oracle(n, H_q, H_kv, D, rd, bs, interleaved, kv, src):
    q, k, v, pos, slots, kc, vc, ks, vs = make(n, H_q, H_kv, D, bs, kv, src, seed=n + rd, pad=2 if n > 4 else 0)
    f = pkv.rotary_frequencies(rd, 10000.0, "by_parts", 8.0, 8192, device=DEV)
    mag = 1.25
    out = pkv.rotary_append(q, k, v, pos, f, slots, kc, vc, ks, vs, magnitude=mag, interleaved=interleaved)
    assert pkv.device_error(DEV) == 0
    p, fr = pos.cpu().numpy(), f.cpu().numpy()

    def bound(x, y):
        # binary32: sine and cosine of an angle off by 2^-24 pi, one factor,
        # one product and one sum: less than 2^-20 of the pair's sizes
        a = np.abs(x)
        s = a.copy()
        if interleaved:
            s[..., 0:rd:2] += a[..., 1:rd:2]
            s[..., 1:rd:2] += a[..., 0:rd:2]
        else:
            s[..., :rd // 2] += a[..., rd // 2:rd]
            s[..., rd // 2:rd] += a[..., :rd // 2]
        return 2.0 ** -20 * mag * s

    qf, kf = q.double().cpu().numpy(), k.double().cpu().numpy()
    want = OC.rotate(qf, p, fr, interleaved, mag)
    got = out.double().cpu().numpy()
    assert (np.abs(got - want) <= 2.0 ** -8 * np.abs(want) * 1.01 + bound(qf, want)).all()
    if src == "bf16":
        assert torch.equal(out[..., rd:], q[..., rd:])

    live = (slots >= 0).cpu().numpy()
    sl = slots[slots >= 0]
    want = OC.rotate(kf, p, fr, interleaved, mag)[live]
    b = bound(kf[live], want)
    if kv == "bf16":
        got = rows_of(kc, sl).double().cpu().numpy()
        assert (np.abs(got - want) <= 2.0 ** -8 * np.abs(want) * 1.01 + b).all()
        assert torch.equal(rows_of(vc, sl), v[slots >= 0].to(torch.bfloat16))
    else:
        s = ks.double().cpu().numpy()[live][:, :, None]
        got = rows_of(kc, sl).view(torch.float8_e4m3fn).double().cpu().numpy() * s
        lim = np.clip(want, -448 * s, 448 * s)
        # half a step: 2^-4 of a normal code, 2^-10 below 2^-6
        tol = np.maximum(2.0 ** -4 * np.abs(lim), 2.0 ** -10 * s) * 1.01 + b
        assert (np.abs(got - lim) <= tol).all()
    # slots no token names keep what they held
    used = torch.zeros(kc.shape[0] * bs, dtype=torch.bool, device=DEV)
    used[sl] = True
    rest = (~used).nonzero().flatten()
    assert torch.all(rows_of(kc, rest) == 7) and torch.all(rows_of(vc, rest) == 7)


@pytest.mark.parametrize("kv,src", [("bf16", "bf16"), ("bf16", "f32"), ("e4m3", "bf16"), ("e4m3", "f32")])
def test_angle_zero_is_append_bit_for_bit(kv, src):
    q, k, v, pos, slots, kc, vc, ks, vs = make(300, 4, 2, 128, 16, kv, src)
    kc2, vc2 = kc.clone(), vc.clone()
    f = torch.zeros(64, dtype=torch.float64, device=DEV)
    out = pkv.rotary_append(q, k, v, pos, f, slots, kc, vc, ks, vs)
    pkv.append(k, v, slots, kc2, vc2, ks, vs)
    assert torch.equal(out, q.to(torch.bfloat16))
    assert torch.equal(kc.view(torch.uint8), kc2.view(torch.uint8))
    assert torch.equal(vc.view(torch.uint8), vc2.view(torch.uint8))


def test_in_place_and_slices_of_a_fused_projection():
    n, hq, hkv, d = 333, 8, 2, 128
    g = torch.Generator(device=DEV).manual_seed(3)
    qkv = torch.randn((n, (hq + 2 * hkv) * d + 64), generator=g, device=DEV).to(torch.bfloat16)
    q = qkv[:, :hq * d].view(n, hq, d)
    k = qkv[:, hq * d:(hq + hkv) * d].view(n, hkv, d)
    v = qkv[:, (hq + hkv) * d:(hq + 2 * hkv) * d].view(n, hkv, d)
    _, _, _, pos, slots, kc, vc, _, _ = make(n, hq, hkv, d, 16, "bf16", "bf16")
    kc2, vc2 = kc.clone(), vc.clone()
    f = pkv.rotary_frequencies(d, device=DEV)
    rest = qkv[:, hq * d:].clone()
    want = pkv.rotary_append(q.contiguous(), k.contiguous(), v.contiguous(), pos, f, slots, kc2, vc2)
    got = pkv.rotary_append(q, k, v, pos, f, slots, kc, vc, out=q)
    assert got.data_ptr() == qkv.data_ptr()
    assert torch.equal(got, want) and torch.equal(kc, kc2) and torch.equal(vc, vc2)
    assert torch.equal(qkv[:, hq * d:], rest)


def test_slots_past_the_cache_are_recorded_and_skipped():
    q, k, v, pos, slots, kc, vc, ks, vs = make(6, 4, 2, 128, 16, "bf16", "bf16")
    slots[2] = kc.shape[0] * 16
    before = kc.clone()
    f = pkv.rotary_frequencies(128, device=DEV)
    out = pkv.rotary_append(q, k, v, pos, f, slots, kc, vc)
    assert pkv.device_error(DEV) == 4
    assert torch.isfinite(out.float()).all()
    changed = (kc != before).any(dim=3).any(dim=1).sum().item()
    assert changed == 5


def test_captured_and_on_another_stream():
    q, k, v, pos, slots, kc, vc, _, _ = make(40, 8, 2, 128, 16, "bf16", "bf16")
    f = pkv.rotary_frequencies(128, device=DEV)
    kc2, vc2 = kc.clone(), vc.clone()
    want = pkv.rotary_append(q, k, v, pos, f, slots, kc2, vc2)
    out = torch.empty_like(want)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        pkv.rotary_append(q, k, v, pos, f, slots, kc, vc, out=out)
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        g.replay()
    s.synchronize()
    assert torch.equal(out, want) and torch.equal(kc, kc2) and torch.equal(vc, vc2)
