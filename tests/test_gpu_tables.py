"""extend_tables and truncate_tables against the one-token-at-a-time model, and
a serving run of tables, rotary append, attention over an E2M1 cache and
truncation, captured in a graph."""

import numpy as np
import pytest
import torch

import paged_kv_cache_222_gb300 as pkv
from oracle import formats as F
from oracle import tables as OT

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda", 0)


def up(x, dt=torch.int32):
    return torch.as_tensor(np.asarray(x)).to(dt).to(DEV)


def cache_of(nb, bs):
    return torch.empty((nb, 1, bs, 64), dtype=torch.uint8, device=DEV)


def make(past, new, bs, spare=9, seed=1, width=0):
    """Tables of the held tokens over a shuffled pool, junk past them; the stack of the rest."""
    rng = np.random.default_rng(seed)
    have = [-(-p // bs) for p in past]
    need = sum(-(-(p + n) // bs) - h for p, n, h in zip(past, new, have))
    nb = sum(have) + need + spare
    perm = rng.permutation(nb).astype(np.int32)
    mb = max([width, 1] + [-(-(p + n) // bs) for p, n in zip(past, new)])
    table = rng.integers(-5, nb + 5, (len(past), mb)).astype(np.int32)
    at = 0
    for b, h in enumerate(have):
        table[b, :h] = perm[at:at + h]
        at += h
    return table, perm[at:].copy(), nb


def check_extend(table, past, new, free, count, bs, nb, most, error=0):
    want = OT.extend(table, past, new, free, count, bs, most, nb)
    t, p, f, c = up(table), up(past), up(free), up([count])
    x = pkv.extend_tables(t, p, up(new), f, c, cache_of(nb, bs), most)
    assert pkv.device_error(DEV) == error and want[8] == (error == 0)
    got = (t, x.context_lens, x.q_starts, x.slot_mapping, x.positions, x.block_starts)
    for g, w in zip(got, want):
        assert np.array_equal(g.cpu().numpy(), w)
    assert x.free_count.item() == want[6] and x.lacking.item() == want[7]
    assert torch.equal(p, up(past)) and torch.equal(f, up(free)) and c.item() == count  # arguments stay
    return x, t


@pytest.mark.parametrize("bs", [16, 32])
@pytest.mark.parametrize("pad", [0, 1, 77])
@pytest.mark.parametrize("past,new", [
    ([0], [1]), ([15], [1]), ([16], [1]), ([0], [0]), ([31, 0, 5], [1, 64, 0]), ([0] * 40, [1] * 40),
    ([0, 0, 7, 0], [0, 0, 300, 0]), ([100] * 3, [0, 0, 0]), ([1, 2, 3, 4, 5], [2500, 1, 0, 31, 1000]), ([], []),
])
def test_extend(past, new, pad, bs):
    table, free, nb = make(past, new, bs)
    check_extend(table, past, new, free, len(free), bs, nb, sum(new) + pad)


@pytest.mark.parametrize("B,hi,most_new,zero", [(256, 8191, 1, 0.0), (700, 300, 3, 0.4), (1500, 100, 40, 0.9),
                                                (33, 4000, 2000, 0.2), (2100, 50, 1, 0.99), (1024, 64, 16, 0.0)])
def test_extend_many(B, hi, most_new, zero):
    rng = np.random.default_rng(B)
    past, new = rng.integers(0, hi, B), rng.integers(1, most_new + 1, B)
    new[rng.random(B) < zero] = 0
    table, free, nb = make(past.tolist(), new.tolist(), 16, seed=B)
    check_extend(table, past, new, free, len(free), 16, nb, int(new.sum()) + 40)
    # exactly as many blocks as it takes; then one fewer
    need = int((-(-(past + new) // 16) - -(-past // 16)).sum())
    check_extend(table, past, new, free, need, 16, nb, int(new.sum()))
    if need:
        x, t = check_extend(table, past, new, free, need - 1, 16, nb, int(new.sum()))
        assert x.lacking.item() == 1 and torch.all(x.slot_mapping == -1) and torch.equal(t, up(table))


def test_the_largest_batch():
    B = 65535
    rng = np.random.default_rng(3)
    past, new = rng.integers(0, 40, B), (rng.random(B) < 0.5).astype(np.int64)
    table, free, nb = make(past.tolist(), new.tolist(), 32, seed=3)
    check_extend(table, past, new, free, len(free), 32, nb, int(new.sum()) + 5)


def test_a_long_prompt():
    past, new = [0, 131071, 0], [131072, 1, 5]
    table, free, nb = make(past, new, 16, seed=5)
    check_extend(table, past, new, free, len(free), 16, nb, sum(new) + 3)


def test_what_is_refused_on_the_device():
    past, new = [10, 20, 30, 40], [5, 6, 7, 8]
    table, free, nb = make(past, new, 16, seed=6)
    n = len(free)
    for b, p, k in ((0, -1, 5), (1, 20, -1), (2, 30, 10 ** 6), (3, 2 ** 31 - 1, 1), (3, 2 ** 31 - 1, 2 ** 31 - 1)):
        pp, kk = list(past), list(new)
        pp[b], kk[b] = p, k
        check_extend(table, pp, kk, free, n, 16, nb, 60, error=3)
    check_extend(table, past, new, free, n, 16, nb, sum(new) - 1, error=3)     # more tokens than places
    check_extend(table, past, new, free, -1, 16, nb, 60, error=2)              # counts that are none
    check_extend(table, past, new, free, n + 1, 16, nb, 60, error=2)
    for bad in (-1, nb, 2 ** 31 - 1):                                          # bad ids on the stack, in the table
        f = free.copy()
        f[n - 1] = bad
        # request 0 asks for more than its table's three entries: refused before any id is looked at
        check_extend(table, past, [40, 6, 7, 8], f, n, 16, nb, 80, error=3)
        check_extend(table, past, [30, 6, 7, 8], f, n, 16, nb, 80, error=2)
        t = table.copy()
        t[2, 1] = bad
        check_extend(t, past, new, free, n, 16, nb, 60, error=2)


@pytest.mark.parametrize("bs", [16, 32])
@pytest.mark.parametrize("ctx,keep", [
    ([1], [0]), ([16], [16]), ([17], [16]), ([0], [0]), ([100, 0, 33, 64], [0, 0, 32, 17]), ([], []),
    ([5000, 3, 20000], [4999, 0, 0]), ([40] * 500, [8] * 500),
])
def test_truncate(ctx, keep, bs):
    table, free, nb = make(ctx, [0] * len(ctx), bs, seed=7)
    full = np.concatenate([free, np.full(nb - len(free), -9, dtype=np.int32)])
    check_truncate(table, ctx, keep, full, len(free), bs, nb)


def check_truncate(table, ctx, keep, free, count, bs, nb, error=0):
    want, n, good = OT.truncate(table, ctx, keep, free, count, bs, nb)
    t, f, c = up(table), up(free), up([count])
    got = pkv.truncate_tables(t, up(ctx), up(keep), f, c, cache_of(nb, bs))
    assert pkv.device_error(DEV) == error and good == (error == 0)
    assert got.item() == n and c.item() == count
    assert np.array_equal(f.cpu().numpy(), want) and torch.equal(t, up(table))


def test_truncate_many():
    rng = np.random.default_rng(8)
    ctx = rng.integers(0, 3000, 1300)
    keep = (ctx * rng.random(1300)).astype(np.int64)
    keep[rng.random(1300) < 0.3] = 0
    table, free, nb = make(ctx.tolist(), [0] * 1300, 16, seed=8)
    full = np.concatenate([free, np.full(nb - len(free), -9, dtype=np.int32)])
    check_truncate(table, ctx, keep, full, len(free), 16, nb)
    need = int((-(-ctx // 16) - -(-keep // 16)).sum())
    check_truncate(table, ctx, keep, full[:5 + need], 5, 16, nb)               # they just fit
    check_truncate(table, ctx, keep, full[:5 + need], 6, 16, nb, error=2)      # they do not
    check_truncate(table, ctx, keep, full, -1, 16, nb, error=2)


def test_truncate_refuses_on_the_device():
    ctx, keep = [100, 50, 70], [10, 20, 30]
    table, free, nb = make(ctx, [0] * 3, 16, seed=9)
    full = np.concatenate([free, np.full(nb - len(free), -9, dtype=np.int32)])
    for b, c, k in ((0, 100, -1), (1, 50, 51), (2, 10 ** 6, 30), (2, -1, -1)):
        cc, kk = list(ctx), list(keep)
        cc[b], kk[b] = c, k
        check_truncate(table, cc, kk, full, len(free), 16, nb, error=3)
    for bad in (-1, nb):
        t = table.copy()
        t[0, 5] = bad
        check_truncate(t, ctx, keep, full, len(free), 16, nb, error=2)


def test_in_place_and_undone():
    past, new = [10, 0, 33, 64], [100, 5, 0, 1]
    table, free, nb = make(past, new, 16, seed=10)
    t, lens, f, c, cache = up(table), up(past), up(free), up([len(free)]), cache_of(nb, 16)
    x = pkv.extend_tables(t, lens, up(new), f, c, cache, 120)
    out = pkv.ExtendedTables(lens, *(torch.empty_like(y) for y in x[1:5]), c, torch.empty_like(x.lacking))
    t2 = up(table)
    y = pkv.extend_tables(t2, lens, up(new), f, c, cache, 120, out=out)
    assert y is out and torch.equal(t, t2)
    for a, b in zip(x, y):
        assert torch.equal(a, b)
    assert lens.tolist() == [110, 5, 33, 65]
    assert pkv.truncate_tables(t2, lens, up(past), f, c, cache, out=c) is c
    assert c.item() == len(free) and torch.equal(f, up(free)) and pkv.device_error(DEV) == 0


def test_refusals():
    past, new = [10, 0], [1, 1]
    table, free, nb = make(past, new, 16, width=3)   # (of one column, the transposed table below would be dense too)
    t, p, n, f, c, cache = up(table), up(past), up(new), up(free), up([len(free)]), cache_of(nb, 16)
    for bad in ((t.long(), p, n, f, c, cache, 8), (t[0], p, n, f, c, cache, 8), (t, p[:1], n, f, c, cache, 8),
                (t, p, n.long(), f, c, cache, 8), (t, p, n, f, up([1, 2]), cache, 8), (t, p, n, f, c, cache[0], 8),
                (t, p, n.cpu(), f, c, cache, 8), (t, p, n, f, c, cache, -1), (t, p, n, f, c, cache, 1.5),
                (t.T.contiguous().T, p, n, f, c, cache, 8), (t, p, n, f[:, None], c, cache, 8)):
        with pytest.raises((TypeError, ValueError)):
            pkv.extend_tables(*bad)
    x = pkv.extend_tables(t, p, n, f, c, cache, 8)
    for out in (x[:6], x._replace(q_starts=x.q_starts[:2]), x._replace(slot_mapping=x.slot_mapping.int()),
                x._replace(positions=x.positions[:4])):
        with pytest.raises((TypeError, ValueError)):
            pkv.extend_tables(t, p, n, f, c, cache, 8, out=out)
    for bad in ((t, p, n[:1], f, c, cache), (t, p, n, f.long(), c, cache), (t, p, n, f, c[:0], cache)):
        with pytest.raises((TypeError, ValueError)):
            pkv.truncate_tables(*bad)
    with pytest.raises((TypeError, ValueError)):
        pkv.truncate_tables(t, p, n, f, c, cache, out=c.long())


def test_on_another_stream():
    past, new = list(range(60)), [3] * 60
    table, free, nb = make(past, new, 16, seed=12)
    want = OT.extend(table, past, new, free, len(free), 16, 5000, nb)
    s = torch.cuda.Stream()
    args = [up(x) for x in (table, past, new, free, [len(free)])]
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        x = pkv.extend_tables(*args, cache_of(nb, 16), 5000)
        n = pkv.truncate_tables(args[0], x.context_lens, args[1], args[3], x.free_count, cache_of(nb, 16))
    s.synchronize()
    assert np.array_equal(x.slot_mapping.cpu().numpy(), want[3]) and n.item() == len(free)


# ---------------------------------------------------------------- a serving run

def attend_plain(q, K, V, scale):
    """Float64 attention of the last len(q) tokens over K, V [T, H, D]."""
    n, H_q, D = q.shape
    T, H, _ = K.shape
    out = np.zeros((n, H_q, D))
    for i in range(n):
        seen = T - n + i + 1
        for h in range(H_q):
            z = K[:seen, h * H // H_q] @ q[i, h] * scale
            w = np.exp(z - z.max())
            out[i, h] = (w / w.sum()) @ V[:seen, h * H // H_q]
    return out


@pytest.mark.parametrize("captured", [False, True])
def test_a_serving_run(captured):
    """Prompts of images and text, then decode steps and rejected drafts, all
    lengths on the GPU: tables, rotary append with three axes into an E2M1
    cache, attention over it, truncation.  Every step's output against a float64
    attention over what the cache holds, read back."""
    B, H_q, H, D, bs, nb, MB, T = 3, 8, 2, 128, 16, 40, 12, 96
    g = torch.Generator(device=DEV).manual_seed(21)
    kc, vc = (pkv.e2m1_cache(nb, H, bs, D) for _ in range(2))
    table = torch.full((B, MB), -1, dtype=torch.int32, device=DEV)
    free = torch.randperm(nb, generator=g, device=DEV).to(torch.int32)
    lens, count = torch.zeros(B, dtype=torch.int32, device=DEV), torch.full((1,), nb, dtype=torch.int32, device=DEV)
    new, keep = torch.zeros_like(lens), torch.zeros_like(lens)
    f, axes = pkv.rotary_frequencies(D, device=DEV), pkv.rotary_axes((16, 24, 24), device=DEV)
    q, k, v = (torch.randn((T, h, D), generator=g, device=DEV).bfloat16() for h in (H_q, H, H))
    grid = torch.zeros((3, T), dtype=torch.int64, device=DEV)
    step = pkv.ExtendedTables(lens, *(torch.zeros(n, dtype=d, device=DEV) for n, d in (
        (B + 1, torch.int32), (T, torch.int64), (T, torch.int64), (B + 1, torch.int32))), count,
        torch.zeros(1, dtype=torch.int32, device=DEV))
    turned, out = torch.empty_like(q), torch.empty_like(q)
    ws = torch.empty(32 << 20, dtype=torch.uint8, device=DEV)

    def forward():
        pkv.extend_tables(table, lens, new, free, count, kc, T, out=step)
        pkv.rotary_append(q, k, v, grid, f, step.slot_mapping, kc, vc, out=turned, axes=axes)
        pkv.chunk_attention(turned, kc, vc, table, lens, step.q_starts, D ** -0.5, max_q_len=T, max_context_len=MB * bs,
                            out=out, workspace=ws)
        pkv.truncate_tables(table, lens, keep, free, count, kc, out=count)

    graph = None
    if captured:
        keep.zero_()
        forward()                                    # (no tokens: nothing happens)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            forward()
    held = [[] for _ in range(B)]                    # the model's tables
    for n_new, n_back in (([40, 1, 17], [0, 0, 0]), ([1, 1, 1], [0, 0, 0]), ([4, 0, 5], [3, 0, 5]), ([1, 60, 2], [0, 9, 0]),
                          ([1, 1, 1], [42, 0, 0])):
        before = lens.tolist()
        new.copy_(up(n_new))
        after = [a + n for a, n in zip(before, n_new)]
        kept = [a - m for a, m in zip(after, n_back)]
        keep.copy_(up(kept))
        for x in (q, k, v):
            x.copy_(torch.randn(x.shape, generator=g, device=DEV))
        at = np.concatenate([np.arange(a, a + n) for a, n in zip(before, n_new)] + [np.zeros(T, dtype=np.int64)])[:T]
        grid.copy_(torch.as_tensor(np.stack([at, at // 7, at % 7])))
        out.fill_(5.0)
        graph.replay() if captured else forward()
        torch.cuda.synchronize()
        assert pkv.device_error(DEV) == 0 and step.lacking.item() == 0
        assert lens.tolist() == after
        tbl = table.cpu().numpy()
        starts = np.concatenate([[0], np.cumsum(n_new)])
        assert step.q_starts.tolist() == starts.tolist()
        blocks = [tbl[b, :-(-after[b] // bs)].tolist() for b in range(B)]
        assert len(set(sum(blocks, []))) == sum(map(len, blocks))            # no block twice
        for b in range(B):
            assert blocks[b][:len(held[b])] == held[b]
            slots = [blocks[b][p // bs] * bs + p % bs for p in range(after[b])]
            assert step.slot_mapping[starts[b]:starts[b + 1]].tolist() == slots[before[b]:]
            if not n_new[b]:
                continue
            K, V = (x.double().cpu().numpy() for x in pkv.read_tokens(up(slots, torch.int64), kc, vc, dtype=torch.float32))
            qb = turned[starts[b]:starts[b + 1]].double().cpu().numpy()
            want = attend_plain(qb, K, V, D ** -0.5)
            scale = attend_plain(qb, K, np.abs(V), D ** -0.5)
            got = out[starts[b]:starts[b + 1]].double().cpu().numpy()
            # output bf16, weights f16, binary32 scores (2^-10 of a weight)
            assert (np.abs(got - want) <= 2.0 ** -8 * 1.01 * np.abs(want) + (2.0 ** -11 + 2.0 ** -10) * scale
                    + 2.0 ** -25 * np.abs(V).sum(0).repeat(H_q // H, 0)).all()
        assert torch.all(out[starts[-1]:] == 5.0)
        # the stack: what the requests do not hold, each once
        held = [blocks[b][:-(-kept[b] // bs)] for b in range(B)]
        n = count.item()
        assert n == nb - sum(map(len, held))
        assert sorted(free[:n].tolist() + sum(held, [])) == list(range(nb))
        lens.copy_(keep)                             # the next step's past


@pytest.mark.parametrize("most", [1 << 31, 1 << 62, -1])
def test_more_tokens_than_a_call_takes_are_refused_before_memory_is_taken(most):
    table, free, nb = make([10], [1], 16)
    t, p, n, f, c, cache = up(table), up([10]), up([1]), up(free), up([len(free)]), cache_of(nb, 16)
    held = torch.cuda.memory_allocated()
    with pytest.raises(ValueError):
        pkv.extend_tables(t, p, n, f, c, cache, most)
    assert torch.cuda.memory_allocated() == held
