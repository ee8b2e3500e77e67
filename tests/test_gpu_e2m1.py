"""GPU parity of E2M1 caches with the oracle: append, read_tokens, block
copies, compaction, and rotary_append into them."""

import numpy as np
import pytest
import torch

import paged_kv_cache_222_gb300 as pkv
from oracle import chunk as OC
from oracle import formats as F

from . import e2m1_support as E

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda", 0)


def rows(n, H, D, src, seed=1):
    g = torch.Generator(device=DEV).manual_seed(seed)
    dt = torch.bfloat16 if src == "bf16" else torch.float32
    x = torch.randn((n, H, D), generator=g, device=DEV) * (1 + 7 * (torch.rand((H, D), generator=g, device=DEV) > 0.95))
    return x.to(dt)


def caches(blocks, H, bs, D, seed=2):
    g = torch.Generator(device=DEV).manual_seed(seed)
    shape = (blocks, H, bs, D // 2 + D // 16)
    return [torch.randint(0, 256, shape, generator=g, device=DEV, dtype=torch.uint8) for _ in range(2)]


def shuffled(n, blocks, bs, pad=0, seed=3):
    g = torch.Generator(device=DEV).manual_seed(seed)
    s = torch.randperm(blocks * bs, generator=g, device=DEV)[:n]
    if pad:
        s[-pad:] = -1
    return s


def expect(cache, x, slots, scale):
    """The cache's (codes, scales) by slot after the rows went in."""
    codes, sc = (a.copy() for a in E.token_bytes(cache))
    c, s = F.e2m1_rows(x.float().cpu().numpy(), None if scale is None else scale.cpu().numpy())
    sl = slots.cpu().numpy()
    codes[sl[sl >= 0]], sc[sl[sl >= 0]] = c[sl >= 0], s[sl >= 0]
    return codes, sc


def same(cache, want):
    got = E.token_bytes(cache)
    return (got[0] == want[0]).all() and (got[1] == want[1]).all()


@pytest.mark.parametrize("src", ["bf16", "f32"])
@pytest.mark.parametrize("scaled", ["no", "heads", "rows"])
@pytest.mark.parametrize("n,H,D,bs", [(1, 1, 64, 16), (37, 3, 128, 16), (500, 8, 128, 32), (300, 5, 64, 32)])
def test_append_bit_for_bit(n, H, D, bs, scaled, src):
    blocks = -(-n // bs) + 2
    k, v = rows(n, H, D, src, 4), rows(n, H, D, src, 5)
    kc, vc = caches(blocks, H, bs, D)
    slots = shuffled(n, blocks, bs, pad=3 if n > 8 else 0)
    ks = vs = None
    if scaled != "no":
        g = torch.Generator(device=DEV).manual_seed(6)
        ks, vs = ((0.3 + torch.rand((n, H) if scaled == "rows" else (H,), generator=g, device=DEV)) / 5 for _ in range(2))
    wk, wv = expect(kc, k, slots, ks), expect(vc, v, slots, vs)
    pkv.append(k, v, slots, kc, vc, ks, vs)
    assert pkv.device_error(DEV) == 0
    assert same(kc, wk) and same(vc, wv)


@pytest.mark.parametrize("D,bs", [(64, 16), (128, 32)])
def test_values_where_rounding_goes_wrong(D, bs):
    x = torch.from_numpy(E.special_rows(D)).to(DEV)[:, None].contiguous()
    n = x.shape[0]
    blocks = -(-n // bs)
    kc, vc = caches(blocks, 1, bs, D)
    slots = shuffled(n, blocks, bs)
    wk, wv = expect(kc, x, slots, None), expect(vc, -x, slots, None)
    pkv.append(x, -x, slots, kc, vc)
    assert same(kc, wk) and same(vc, wv)
    k, v = pkv.read_tokens(slots, kc, vc, dtype=torch.float32)
    want = F.e2m1_values(kc.cpu().numpy()).transpose(0, 2, 1, 3).reshape(-1, 1, D)[slots.cpu().numpy()]
    assert np.array_equal(k.double().cpu().numpy(), want, equal_nan=True) and np.isnan(want).any()


def test_every_bf16_magnitude():
    # one value per group beside a largest one of every scale mantissa: every
    # bf16 in reach of the codes, against the oracle's distances
    top = torch.tensor([6.0 * (8 + m) / 8 for m in range(8)])
    u = torch.arange(0x3C00, 0x40D0, dtype=torch.int32).to(torch.int16).view(torch.bfloat16).float()
    x = torch.zeros((8, u.numel(), 16))
    x[..., 0], x[..., 1] = top[:, None], u
    x[..., 2] = -u
    x = x.reshape(-1, 64).bfloat16().to(DEV)[:, None].contiguous()
    bs, n = 32, x.shape[0]
    kc, vc = caches(-(-n // bs), 1, bs, 64)
    slots = torch.arange(n, device=DEV)
    w = expect(kc, x, slots, None)
    pkv.append(x, x, slots, kc, vc)
    assert same(kc, w)


@pytest.mark.parametrize("kv", ["bf16", "e4m3", "e2m1"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("H,D,bs", [(3, 128, 16), (8, 64, 32), (1, 64, 16)])
def test_read_tokens(kv, dtype, H, D, bs):
    blocks, n = 9, 77
    g = torch.Generator().manual_seed(7)
    if kv == "bf16":
        kc, vc = (torch.randn((blocks, H, bs, D), generator=g).bfloat16().to(DEV) for _ in range(2))
        vals = [c.double().cpu().numpy() for c in (kc, vc)]
    elif kv == "e4m3":
        kc, vc = ((torch.randn((blocks, H, bs, D), generator=g) * 64).to(torch.float8_e4m3fn).to(DEV) for _ in range(2))
        vals = [F.e4m3_to_f64(c.view(torch.uint8).cpu().numpy()) for c in (kc, vc)]
    else:
        kc, vc = (E.pool(g, blocks, H, bs, D).to(DEV) for _ in range(2))
        vals = [F.e2m1_values(c.cpu().numpy()) for c in (kc, vc)]
    slots = torch.randint(0, blocks * bs, (n,), generator=g).to(DEV)   # the same slot more than once
    slots[5], slots[11] = -1, -7
    for scaled in ((False,) if kv == "bf16" else (True,) if kv == "e4m3" else (False, True)):
        ks = vs = None
        if scaled:
            ks, vs = ((0.5 + torch.rand((n, H), generator=g)).to(DEV) for _ in range(2))
        got = pkv.read_tokens(slots, kc, vc, ks, vs, dtype=dtype)
        assert pkv.device_error(DEV) == 0
        for x, val, s in zip(got, vals, (ks, vs)):
            assert x.shape == (n, H, D) and x.dtype == dtype
            sl = slots.cpu().numpy()
            want = val.transpose(0, 2, 1, 3).reshape(-1, H, D)[np.maximum(sl, 0)]
            want = np.where((sl >= 0)[:, None, None], want, 0.0)
            if s is not None:
                want = want * s.double().cpu().numpy()[..., None]
            # one rounding in binary32, one to bf16
            tol = 2.0 ** -24 + (2.0 ** -8 if dtype == torch.bfloat16 else 0.0)
            assert (np.abs(x.double().cpu().numpy() - want) <= tol * 1.01 * np.abs(want)).all()
    if kv == "bf16" and dtype == torch.bfloat16:  # bit for bit, NaN payloads too
        kc.view(torch.int16)[0, 0, 0, 0] = 0x7FA5
        k, _ = pkv.read_tokens(torch.zeros(1, dtype=torch.int64, device=DEV), kc, vc)
        assert k.view(torch.int16)[0, 0, 0] == 0x7FA5


def test_bad_slots_are_recorded():
    kc, vc = caches(4, 2, 16, 128)
    k = rows(3, 2, 128, "bf16")
    slots = torch.tensor([0, 64, 5], device=DEV)
    wk, wv = expect(kc, k[[0, 2]], slots[[0, 2]], None), expect(vc, k[[0, 2]], slots[[0, 2]], None)
    pkv.append(k, k, slots, kc, vc)
    assert pkv.device_error(DEV) == 4
    assert same(kc, wk) and same(vc, wv)
    x, y = pkv.read_tokens(slots, kc, vc)
    assert pkv.device_error(DEV) == 4
    assert not x[1].any() and not y[1].any() and x[0].any() and x[2].any()


def test_empty_calls():
    kc, vc = caches(4, 2, 16, 128)
    before = kc.clone()
    none = torch.empty(0, dtype=torch.int64, device=DEV)
    pkv.append(rows(0, 2, 128, "f32"), rows(0, 2, 128, "f32"), none, kc, vc)
    k, v = pkv.read_tokens(none, kc, vc)
    assert k.shape == v.shape == (0, 2, 128) and torch.equal(kc, before)


def test_refusals():
    kc, vc = caches(4, 2, 16, 128)
    k, slots = rows(3, 2, 128, "bf16"), torch.arange(3, device=DEV)
    one = torch.ones((3, 2), device=DEV)
    for args in ((k[:, :1], k[:, :1], slots, kc, vc), (k, k, slots[:2], kc, vc), (k, k, slots, kc, vc, one),
                 (k, k, slots, kc, vc, one[:2], one[:2]), (k, k.float(), slots, kc, vc), (k, k, slots.int(), kc, vc),
                 (k.half(), k.half(), slots, kc, vc), (k, k, slots.cpu(), kc, vc),
                 (k.transpose(0, 1).contiguous().transpose(0, 1), k, slots, kc, vc)):
        with pytest.raises((TypeError, ValueError)):
            pkv.append(*args)
    for args in ((slots, kc, vc, one), (slots[:, None], kc, vc), (slots.int(), kc, vc), (slots.cpu(), kc, vc)):
        with pytest.raises((TypeError, ValueError)):
            pkv.read_tokens(*args)
    q = rows(1, 8, 128, "bf16")
    with pytest.raises(pkv.PkvError, match="pkv_chunk_attention"):
        pkv.decode_attention(q, kc, vc, torch.zeros((1, 4), dtype=torch.int32, device=DEV),
                             torch.ones(1, dtype=torch.int32, device=DEV), 0.1)


def test_on_another_stream_and_captured():
    k, v = rows(40, 2, 128, "bf16", 8), rows(40, 2, 128, "bf16", 9)
    kc, vc = caches(4, 2, 16, 128)
    slots = shuffled(40, 4, 16)
    wk = expect(kc, k, slots, None)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        a, b = kc.clone(), vc.clone()
        pkv.append(k, v, slots, a, b)
        x, y = pkv.read_tokens(slots, a, b)
    torch.cuda.current_stream().wait_stream(s)
    assert same(a, wk)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pkv.append(k, v, slots, kc, vc)
        gx, gy = pkv.read_tokens(slots, kc, vc)
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    assert same(kc, wk) and torch.equal(gx, x) and torch.equal(gy, y)
    k.copy_(-k)                                    # other rows in the same place
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(gx, -x)


# ---------------------------------------------------------------- copies and compaction

@pytest.mark.parametrize("D,bs", [(64, 16), (128, 16), (64, 32), (128, 32)])
def test_block_copies(D, bs):
    kc, vc = caches(12, 3, bs, D)
    k0, v0 = kc.clone(), vc.clone()
    pkv.copy_blocks(kc, vc, [1, 4, 7], [2, 11, 0])
    assert pkv.device_error(DEV) == 0
    for c, c0 in ((kc, k0), (vc, v0)):
        w = c0.clone()
        w[[2, 11, 0]] = c0[[1, 4, 7]]
        assert torch.equal(c, w)
    hk, hv = pkv.host_pool_like(kc, 5)
    hk.zero_(), hv.zero_()
    pkv.copy_blocks_between(kc, vc, hk, hv, [3, 8], [4, 0])
    torch.cuda.synchronize()
    assert torch.equal(hk[[4, 0]], kc[[3, 8]].cpu()) and torch.equal(hv[[4, 0]], vc[[3, 8]].cpu())
    assert not hk[[1, 2, 3]].any()


@pytest.mark.parametrize("D,bs,H", [(64, 16, 3), (128, 16, 2), (64, 32, 1), (128, 32, 8)])
def test_compaction(D, bs, H):
    g = torch.Generator().manual_seed(11)
    lens = [700, 1, 40, 333]
    mb = -(-max(lens) // bs)
    pool = sum(-(-n // bs) for n in lens)
    perm = torch.randperm(pool, generator=g).tolist()
    table = np.full((4, mb), -1, dtype=np.int32)
    for b, n in enumerate(lens):
        for j in range(-(-n // bs)):
            table[b, j] = perm.pop()
    kc, vc = caches(pool, H, bs, D)
    first = [3, 0, 0, 100]
    keep = [sorted(torch.randperm(n - f, generator=g)[: (n - f) * 2 // 3 + 1].add(f).tolist()) for n, f in zip(lens, first)]
    starts = np.concatenate([[0], np.cumsum([len(x) for x in keep])]).astype(np.int32)
    flat = np.concatenate(keep).astype(np.int32)
    want = []
    for c in (kc, vc):
        codes, sc = F.e2m1_unpack(c.cpu().numpy())
        want.append([OC.compact(x, table, flat, starts, first) for x in (codes, sc)])
    up = [torch.from_numpy(x).to(DEV) for x in (table, flat, starts, np.array(first, dtype=np.int32))]
    pkv.compact_tokens(kc, vc, up[0], up[1], up[2], dst_start=up[3])
    assert pkv.device_error(DEV) == 0
    for c, w in zip((kc, vc), want):
        codes, sc = F.e2m1_unpack(c.cpu().numpy())
        assert (codes == w[0]).all() and (sc == w[1]).all()


# ---------------------------------------------------------------- rotary append

@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("scaled", [False, True])
@pytest.mark.parametrize("src", ["bf16", "f32"])
@pytest.mark.parametrize("H_q,H,D,rd,bs", [(8, 2, 128, 128, 16), (5, 1, 64, 64, 32), (3, 3, 128, 64, 16),
                                           (4, 4, 64, 16, 16), (16, 8, 128, 48, 32), (6, 3, 64, 48, 16)])
def test_rotary_append(H_q, H, D, rd, bs, src, scaled, interleaved):
    n, blocks = 333, 30
    q, k, v = rows(n, H_q, D, src, 12), rows(n, H, D, src, 13), rows(n, H, D, src, 14)
    g = torch.Generator(device=DEV).manual_seed(15)
    pos = torch.randint(-1 << 20, 1 << 20, (n,), generator=g, device=DEV)
    kc, vc = caches(blocks, H, bs, D)
    slots = shuffled(n, blocks, bs, pad=2)
    ks = vs = None
    if scaled:
        ks, vs = ((0.5 + torch.rand((n, H), generator=g, device=DEV)) / 8 for _ in range(2))
    wv = expect(vc, v, slots, vs)
    old = E.token_bytes(kc)
    f = pkv.rotary_frequencies(rd, device=DEV)
    # angle zero: what append writes, bit for bit
    a, b = kc.clone(), vc.clone()
    wk = expect(kc, k, slots, ks)
    pkv.rotary_append(q, k, v, pos, torch.zeros_like(f), slots, a, b, ks, vs, interleaved=interleaved)
    assert same(a, wk) and same(b, wv)
    pkv.rotary_append(q, k, v, pos, f, slots, kc, vc, ks, vs, magnitude=1.25, interleaved=interleaved)
    assert pkv.device_error(DEV) == 0
    assert same(vc, wv)
    # the turned keys: a value near a border may fall on its other side, no more
    live = slots.cpu().numpy() >= 0
    sl = slots.cpu().numpy()[live]
    x = OC.rotate(k.double().cpu().numpy(), pos.cpu().numpy(), f.cpu().numpy(), interleaved, 1.25)[live]
    if scaled:
        x = x / ks.double().cpu().numpy()[live][..., None]
    codes, sc = E.token_bytes(kc)
    wc, ws = F.e2m1_rows(x.astype(np.float32))
    assert (codes[sl] != wc).mean() < 1e-3 and (sc[sl] != ws).mean() < 1e-3
    got = F.E2M1_VALUES[codes[sl]] * np.repeat(F.e4m3_to_f64(sc[sl]), 16, axis=-1)
    # half the widest step, 1, times a scale of at most (largest / 6)(1 + 2^-4)
    amax = np.abs(x).reshape(x.shape[:-1] + (-1, 16)).max(-1, keepdims=True)
    tol = np.broadcast_to(amax / 6 * (1 + 2.0 ** -4) * (1 + 2.0 ** -18), amax.shape[:-1] + (16,)).reshape(x.shape)
    assert (np.abs(got - x) <= tol).all()
    rest = np.setdiff1d(np.arange(blocks * bs), sl)
    assert (codes[rest] == old[0][rest]).all() and (sc[rest] == old[1][rest]).all()
