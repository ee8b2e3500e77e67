"""GPU parity of rotary_append with positions along several axes."""

import numpy as np
import pytest
import torch

import paged_kv_cache_222_gb300 as pkv

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda", 0)


def make(n, H_q, H, D, bs=16, src="bf16", seed=1, far=1 << 16, axes=3):
    g = torch.Generator(device=DEV).manual_seed(seed)
    dt = torch.bfloat16 if src == "bf16" else torch.float32
    q, k, v = (torch.randn((n, h, D), generator=g, device=DEV).to(dt) for h in (H_q, H, H))
    blocks = -(-max(n, 1) // bs) + 2
    kc, vc = (torch.zeros((blocks, H, bs, D), dtype=torch.bfloat16, device=DEV) for _ in range(2))
    pos = torch.randint(-far, far, (axes, n), generator=g, device=DEV)
    return q, k, v, pos, torch.randperm(blocks * bs, generator=g, device=DEV)[:n], kc, vc


def turned(x, pos, axes, f, interleaved, mag):
    """Float64, pair by pair, and the bound of binary32 arithmetic."""
    x, pos, axes, f = x.double().cpu().numpy(), pos.cpu().numpy(), axes.cpu().numpy(), f.cpu().numpy()
    y, tol = x.copy(), np.zeros_like(x)
    half = len(f)
    for i in range(half):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
        angle = pos[axes[i]].astype(np.float64) * f[i]
        z = (x[..., a] + 1j * x[..., b]) * (mag * np.exp(1j * angle))[:, None]
        y[..., a], y[..., b] = z.real, z.imag
        # sine and cosine of an angle off by 2^-24 pi, a factor, a product, a sum
        tol[..., a] = tol[..., b] = 2.0 ** -20 * mag * (np.abs(x[..., a]) + np.abs(x[..., b]))
    return y, tol + 2.0 ** -8 * 1.01 * np.abs(y)


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("mixed", [False, True])
@pytest.mark.parametrize("src", ["bf16", "f32"])
@pytest.mark.parametrize("n,H_q,H,D,cuts", [(1, 4, 1, 64, (16, 8, 8)), (61, 8, 2, 128, (16, 24, 24)),
                                            (300, 5, 5, 128, (1, 62, 1)), (33, 3, 1, 128, (8, 8)),
                                            (40, 2, 1, 64, (4, 4, 4, 4))])
def test_matches_the_definition(n, H_q, H, D, cuts, src, mixed, interleaved):
    q, k, v, pos, slots, kc, vc = make(n, H_q, H, D, src=src, axes=len(cuts))
    f = pkv.rotary_frequencies(2 * sum(cuts), device=DEV)
    axes = pkv.rotary_axes(cuts, mixed=mixed, device=DEV)
    out = pkv.rotary_append(q, k, v, pos, f, slots, kc, vc, magnitude=1.1, interleaved=interleaved, axes=axes)
    assert pkv.device_error(DEV) == 0
    want, tol = turned(q, pos, axes, f, interleaved, 1.1)
    assert (np.abs(out.double().cpu().numpy() - want) <= tol).all()
    got = kc[slots // 16, :, slots % 16]
    want, tol = turned(k, pos, axes, f, interleaved, 1.1)
    assert (np.abs(got.double().cpu().numpy() - want) <= tol).all()
    assert torch.equal(vc[slots // 16, :, slots % 16], v.bfloat16())


def test_one_axis_is_the_plain_call():
    q, k, v, pos, slots, kc, vc = make(50, 4, 2, 128)
    f = pkv.rotary_frequencies(128, device=DEV)
    a = pkv.rotary_append(q, k, v, pos[1].contiguous(), f, slots, kc, vc)
    kc2, vc2 = torch.zeros_like(kc), torch.zeros_like(vc)
    for p, axes in ((pos[1:2], [0] * 64), (pos, [1] * 64), (pos[1].expand(3, 50), [0, 1, 2, 0] * 16)):
        b = pkv.rotary_append(q, k, v, p, f, slots, kc2, vc2, axes=torch.tensor(axes, dtype=torch.int32, device=DEV))
        assert torch.equal(a, b) and torch.equal(kc, kc2)


def test_positions_in_a_wider_buffer():
    q, k, v, pos, slots, kc, vc = make(50, 4, 2, 128)
    f, axes = pkv.rotary_frequencies(128, device=DEV), pkv.rotary_axes((16, 24, 24), device=DEV)
    a = pkv.rotary_append(q, k, v, pos, f, slots, kc, vc, axes=axes)
    wide = torch.full((3, 99), 7, dtype=torch.int64, device=DEV)
    wide[:, 20:70] = pos
    assert torch.equal(pkv.rotary_append(q, k, v, wide[:, 20:70], f, slots, kc, vc, axes=axes), a)


def test_an_axis_that_is_none_leaves_its_pairs():
    q, k, v, pos, slots, kc, vc = make(9, 2, 1, 64)
    f, axes = pkv.rotary_frequencies(64, device=DEV), pkv.rotary_axes((16, 8, 8), device=DEV)
    want = pkv.rotary_append(q, k, v, pos, f, slots, kc, vc, axes=axes)
    for bad in (3, -1, 2 ** 31 - 1, -2 ** 31):
        axes2 = axes.clone()
        axes2[4] = bad
        out = pkv.rotary_append(q, k, v, pos, f, slots, kc, vc, axes=axes2)
        assert pkv.device_error(DEV) == 5
        keep = [i for i in range(64) if i not in (4, 36)]
        assert torch.equal(out[..., keep], want[..., keep]) and torch.equal(out[..., [4, 36]], q[..., [4, 36]])


def test_refusals():
    q, k, v, pos, slots, kc, vc = make(9, 2, 1, 64)
    f, axes = pkv.rotary_frequencies(64, device=DEV), pkv.rotary_axes((16, 8, 8), device=DEV)
    for p, a in ((pos[0], axes), (pos, None), (pos, axes[:5]), (pos, axes.long()), (pos[:, :8], axes),
                 (pos.int(), axes), (pos.cpu(), axes), (pos.T.contiguous().T, axes), (pos, axes.cpu())):
        with pytest.raises((TypeError, ValueError)):
            pkv.rotary_append(q, k, v, p, f, slots, kc, vc, axes=a)
    with pytest.raises(pkv.PkvError):
        pkv.rotary_append(q, k, v, pos[:0], f, slots, kc, vc, axes=axes)


def test_captured():
    q, k, v, pos, slots, kc, vc = make(20, 4, 2, 128)
    f, axes = pkv.rotary_frequencies(128, device=DEV), pkv.rotary_axes((16, 24, 24), mixed=True, device=DEV)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = pkv.rotary_append(q, k, v, pos, f, slots, kc, vc, axes=axes)
    pos.add_(5)
    graph.replay()
    torch.cuda.synchronize()
    kept = kc.clone()
    assert torch.equal(out, pkv.rotary_append(q, k, v, pos, f, slots, kc, vc, axes=axes)) and torch.equal(kc, kept)
