"""GPU parity of compact_tokens (bit for bit), and a serving run that uses the
new operators together."""

import numpy as np
import pytest
import torch

import paged_kv_cache_222_gb300 as pkv
from oracle import chunk as OC

from . import chunk_support as C

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda", 0)


def make(lens, H_kv, D, bs, kv, seed):
    g = torch.Generator().manual_seed(seed)
    nblk = [-(-n // bs) for n in lens]
    pool = sum(nblk) + 3
    perm = torch.randperm(pool, generator=g).numpy().astype(np.int32)
    table = np.full((len(lens), max(max(nblk), 1)), -1, dtype=np.int32)
    at = 0
    for b, n in enumerate(nblk):
        table[b, :n] = perm[at:at + n]
        at += n
    dt = torch.int16 if kv == "bf16" else torch.uint8
    hi = 30000 if kv == "bf16" else 255
    k, v = (torch.randint(0, hi, (pool, H_kv, bs, D), generator=g).to(dt) for _ in range(2))
    return table, k, v


def pick(rng, lens, kind):
    keep, starts, first = [], [0], []
    for n in lens:
        f = 0
        if kind == "half":
            kk = sorted(rng.choice(n, n // 2, replace=False).tolist())
        elif kind == "all":
            kk = list(range(n))
        elif kind == "tail":
            f = n // 3
            kk = list(range(n - n // 4, n)) if n >= 4 else []
        elif kind == "one":
            kk = [n - 1] if n else []
        else:
            kk = []
        keep += kk
        starts.append(len(keep))
        first.append(f)
    return np.array(keep, dtype=np.int32), np.array(starts, dtype=np.int32), np.array(first, dtype=np.int32)


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("H_kv,D,bs", [(1, 64, 16), (2, 128, 16), (8, 128, 32)])
@pytest.mark.parametrize("kind", ["half", "all", "tail", "one"])
def test_matches_oracle(kind, H_kv, D, bs, kv):
    lens = [1, 0, 17, 300, 1030, 64]
    table, k, v = make(lens, H_kv, D, bs, kv, seed=H_kv + D)
    keep, starts, first = pick(np.random.default_rng(7), lens, kind)
    want = [torch.from_numpy(OC.compact(c.numpy(), table, keep, starts, first)) for c in (k, v)]
    dt = torch.bfloat16 if kv == "bf16" else torch.uint8
    kd, vd = k.to(DEV).view(dt), v.to(DEV).view(dt)
    pkv.compact_tokens(kd, vd, torch.from_numpy(table).to(DEV), torch.from_numpy(keep).to(DEV),
                       torch.from_numpy(starts).to(DEV), dst_start=torch.from_numpy(first).to(DEV))
    assert pkv.device_error(DEV) == 0
    assert torch.equal(kd.view(k.dtype).cpu(), want[0]) and torch.equal(vd.view(k.dtype).cpu(), want[1])


def test_any_order_and_repeats_not_before_the_destination():
    table, k, v = make([2000], 2, 128, 16, "bf16", seed=3)
    rng = np.random.default_rng(1)
    keep = np.array([rng.integers(j, 2000) for j in range(1500)], dtype=np.int32)
    starts = np.array([0, 1500], dtype=np.int32)
    want = OC.compact(k.numpy(), table, keep, starts)
    kd, vd = k.to(DEV).view(torch.bfloat16), v.to(DEV).view(torch.bfloat16)
    pkv.compact_tokens(kd, vd, torch.from_numpy(table).to(DEV), torch.from_numpy(keep).to(DEV),
                       torch.from_numpy(starts).to(DEV))
    assert pkv.device_error(DEV) == 0
    assert np.array_equal(kd.view(torch.int16).cpu().numpy(), want)


def test_bad_entries_are_recorded_and_not_moved():
    table, k, v = make([64, 64], 1, 64, 16, "bf16", seed=4)
    t = torch.from_numpy(table).to(DEV)

    def go(keep, starts, **kw):
        kd, vd = k.to(DEV).view(torch.bfloat16), v.to(DEV).view(torch.bfloat16)
        pkv.compact_tokens(kd, vd, t, torch.tensor(keep, dtype=torch.int32, device=DEV),
                           torch.tensor(starts, dtype=torch.int32, device=DEV), **kw)
        return kd.view(torch.int16).cpu(), pkv.device_error(DEV)

    got, err = go([3, 0, 9, 5000, -1], [0, 5, 5])       # entry 1 before its place, 3 past the table, 4 negative
    assert err == 3
    ok = torch.from_numpy(OC.compact(k.numpy(), table, np.array([3, 1, 9]), np.array([0, 3, 3])))
    assert torch.equal(got, ok)
    got, err = go([3, 4], [0, 5, 1])                    # ranges that leave the list
    assert err == 3 and torch.equal(got, k)
    got, err = go([3, 4], [0, 2, 2], max_keep=1)        # longer than the bound
    assert err == 3 and torch.equal(got, k)
    got, err = go([3, 4], [0, 2, 2], dst_start=torch.tensor([-1, 0], dtype=torch.int32, device=DEV))
    assert err == 3 and torch.equal(got, k)


def test_a_serving_run():
    """Prompts, decode steps, an eviction and more steps through rotary_append,
    chunk_attention, compact_tokens and the block manager, against float64."""
    hq, hkv, d, bs = 8, 2, 128, 16
    gen = torch.Generator().manual_seed(11)
    bm = pkv.BlockManager(200, bs)
    kc = torch.zeros((200, hkv, bs, d), dtype=torch.bfloat16, device=DEV)
    vc = torch.zeros_like(kc)
    f = pkv.rotary_frequencies(d, device=DEV)
    ids = [0, 1, 2]
    for i in ids:
        bm.add_sequence(i)
    # what the cache should hold, per sequence: float64 of the bf16 rows
    keys, vals = ([np.zeros((0, hkv, d)) for _ in ids] for _ in range(2))
    seen = [0, 0, 0]  # rotary positions handed out

    def step(n_new, softcap, window):
        T = sum(n_new)
        q, k, v = (torch.randn((T, h, d), generator=gen).to(torch.bfloat16) for h in (hq, hkv, hkv))
        slots, cow = bm.append(ids, n_new)
        assert len(cow) == 0
        pos = np.concatenate([seen[i] + np.arange(n) for i, n in enumerate(n_new)])
        qr = pkv.rotary_append(q.to(DEV), k.to(DEV), v.to(DEV), torch.from_numpy(pos).to(DEV), f,
                               torch.from_numpy(slots).to(DEV), kc, vc)
        table, lens = bm.block_tables(ids, 40)
        starts = np.concatenate([[0], np.cumsum(n_new)]).astype(np.int32)
        out = pkv.chunk_attention(qr, kc, vc, torch.from_numpy(table).to(DEV), torch.from_numpy(lens).to(DEV),
                                  torch.from_numpy(starts).to(DEV), d ** -0.5, max_q_len=max(n_new),
                                  max_context_len=int(lens.max()), softcap=softcap, window=window)
        assert pkv.device_error(DEV) == 0
        kr = OC.rotate(k.double().numpy(), pos, f.cpu().numpy())
        qw = OC.rotate(q.double().numpy(), pos, f.cpu().numpy())
        got = out.double().cpu().numpy()
        for i, n in enumerate(n_new):
            a, b = starts[i], starts[i + 1]
            keys[i] = np.concatenate([keys[i], kr[a:b]])
            vals[i] = np.concatenate([vals[i], v.double().numpy()[a:b]])
            seen[i] += n
            see = OC.visible(len(keys[i]), n, window)
            for h in range(hq):
                K, V = keys[i][:, h // 4], vals[i][:, h // 4]
                z = qw[a:b, h] @ K.T * d ** -0.5
                if softcap:
                    z = softcap * np.tanh(z / softcap)
                # turned queries and keys are rounded to bf16 (2^-8 each): a score moves by
                # 2^-7 sum |q k| scale / sqrt(d)-fold cancelling, at most 2^-7 |q| |k| scale
                dz = 2.0 ** -7 * np.linalg.norm(qw[a:b, h], axis=1)[:, None] * np.linalg.norm(K, axis=1) * d ** -0.5
                z = np.where(see, z, -np.inf)
                p = np.exp(z - z.max(axis=1, keepdims=True))
                p /= p.sum(axis=1, keepdims=True)
                ref = p @ V
                A = p @ np.abs(V)
                # d out = sum p dz (v - out)
                move = (p * dz) @ np.abs(V) + (p * dz).sum(axis=1, keepdims=True) * np.abs(ref)
                tol = 2.0 ** -8 * np.abs(ref) * 1.01 + (2.0 ** -8 + 2.0 ** -10) * A + 1.1 * move
                assert (np.abs(got[a:b, h] - ref) <= tol).all()

    step([70, 1, 200], 0.0, 0)
    step([1, 1, 1], 20.0, 0)
    step([5, 130, 1], 0.0, 64)
    # eviction: the first 4 tokens and a random half of the others stay
    rng = np.random.default_rng(5)
    keep, starts = [], [0]
    for i in ids:
        n = len(keys[i])
        kk = sorted(set(range(4)) | set(rng.choice(n, n // 2, replace=False).tolist()))
        keep += kk
        starts.append(len(keep))
        keys[i], vals[i] = keys[i][kk], vals[i][kk]
    table, _ = bm.block_tables(ids, 40)
    pkv.compact_tokens(kc, vc, torch.from_numpy(table).to(DEV), torch.tensor(keep, dtype=torch.int32, device=DEV),
                       torch.tensor(starts, dtype=torch.int32, device=DEV))
    free = bm.num_free()
    for i in ids:
        bm.truncate(i, starts[i + 1] - starts[i])
    assert bm.num_free() > free
    step([1, 1, 1], 0.0, 0)
    step([33, 1, 2], 30.0, 50)
