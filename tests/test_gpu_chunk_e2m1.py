"""GPU parity of ragged chunk attention over E2M1 caches with the float64 oracle."""

import numpy as np
import pytest
import torch

import paged_kv_cache_222_gb300 as pkv

from . import chunk_support as C
from . import e2m1_support as E

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda", 0)


def run(case, **kw):
    args, kwargs = C.device_args(case, DEV)
    kwargs.update(kw)
    out = pkv.chunk_attention(*args, **kwargs)
    assert pkv.device_error(DEV) == 0
    return out


SINGLE = ([1, 1, 1, 1, 1, 1], [1, 2, 17, 64, 65, 1000])
FEW = ([2, 1, 0, 2, 1, 2, 2, 1], [2, 1, 40, 33, 31, 32, 300, 129])
RAGGED = ([1, 5, 0, 33, 130, 64, 2], [1, 5, 40, 33, 300, 900, 257])
PROMPTS = ([1, 127, 128, 129, 300], [1, 127, 128, 129, 300])
LENS = pytest.mark.parametrize("lens", [SINGLE, FEW, RAGGED, PROMPTS], ids=["single", "few", "ragged", "prompts"])
MOST = pytest.mark.parametrize("lens", [SINGLE, FEW, RAGGED], ids=["single", "few", "ragged"])


@pytest.mark.parametrize("H_q,H_kv,D,bs", [(8, 1, 128, 16), (6, 2, 64, 32), (4, 4, 128, 32), (7, 1, 64, 16),
                                           (16, 1, 128, 16), (5, 1, 128, 32), (24, 2, 64, 16), (9, 3, 64, 32),
                                           (10, 1, 128, 16)])
@LENS
def test_plain_scores(lens, H_q, H_kv, D, bs):
    case = E.chunk_case(*lens, H_q, H_kv, D, bs, scaled=H_q % 2 == 0, seed=H_q * 100 + D)
    E.chunk_check(run(case), case)


MODS = [dict(softcap=5.0), dict(softcap=30.0), dict(softcap=300.0), dict(bias=True), dict(window=1), dict(window=100),
        dict(window=5000), dict(prefix=3), dict(prefix=10 ** 6), dict(window=40, prefix=20),
        dict(window=130, prefix=200, bias=True), dict(softcap=20.0, bias=True, window=77)]


def _with_prefix(mods, n):
    m = dict(mods)
    if "prefix" in m:  # another prefix for every sequence, none for the first
        m["prefix"] = [0] + [m["prefix"] + i for i in range(n - 1)]
    return m


@pytest.mark.parametrize("mods", MODS, ids=[",".join(f"{k}={v}" for k, v in m.items()) for m in MODS])
@MOST
@pytest.mark.parametrize("D,bs", [(64, 16), (128, 16), (128, 32), (64, 32)])
def test_modified_scores(lens, mods, D, bs):
    case = E.chunk_case(*lens, 8, 2, D, bs, seed=77, **_with_prefix(mods, len(lens[0])))
    E.chunk_check(run(case), case)


@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("softcap", [1e-3, 0.5, 1e4, 1e7, 1e30])
@MOST
def test_tiny_and_enormous_caps(lens, softcap, bias):
    case = E.chunk_case(*lens, 8, 2, 128, 16, softcap=softcap, bias=bias, seed=78)
    E.chunk_check(run(case), case)


@pytest.mark.parametrize("split_tokens", [128, 256, 640])
@pytest.mark.parametrize("mods", [{}, dict(window=300), dict(window=200, prefix=129), dict(softcap=9.0, bias=True)],
                         ids=["plain", "window", "window+prefix", "cap+bias"])
@MOST
@pytest.mark.parametrize("D,bs", [(128, 16), (64, 32)])
def test_splits(lens, mods, split_tokens, D, bs):
    case = E.chunk_case(*lens, 8, 1, D, bs, seed=5, **_with_prefix(mods, len(lens[0])))
    E.chunk_check(run(case, split_tokens=split_tokens), case)


@pytest.mark.parametrize("q_lens", [[1] * 4, [2, 1, 2, 2], [40, 3, 200, 1]], ids=["single", "few", "ragged"])
def test_blocks_behind_the_window_may_be_gone(q_lens):
    case = E.chunk_case(q_lens, [700, 333, 512, 650], 8, 2, 128, 16, window=50, prefix=[0, 16, 10, 33], seed=9,
                        free_behind_window=True)
    assert (case["table"][0, :20] == -1).any()
    for st in (0, 128):
        E.chunk_check(run(case, split_tokens=st), case)


@pytest.mark.parametrize("q_lens", [[2, 2, 2], [8, 8, 8], [200, 4, 130]], ids=["few", "some", "many"])
def test_queries_before_position_zero_give_zeros(q_lens):
    ctxs = [5, 0, 8] if q_lens[0] > 5 else [1, 0, 2]
    case = E.chunk_case(q_lens, ctxs, 8, 2, 128, 16, prefix=[3, 3, 3], seed=3)
    out = run(case)
    E.chunk_check(out, case)
    assert torch.all(out[: q_lens[0] - ctxs[0]] == 0)
    assert torch.all(out[q_lens[0]:q_lens[0] + q_lens[1]] == 0)


@pytest.mark.parametrize("q_lens", [[1, 1], [2, 1], [150, 3]], ids=["single", "few", "many"])
def test_rows_behind_the_last_sequence_stay(q_lens):
    case = E.chunk_case(q_lens, [300, 20], 8, 2, 128, 16, tail_rows=7, seed=4)
    out = torch.full_like(case["q"], 3.5, device=DEV)
    assert run(case, out=out) is out
    E.chunk_check(out, case)
    assert torch.all(out[sum(q_lens):] == 3.5)


@MOST
def test_large_and_peaked_scores(lens):
    # queries 30 times larger: binary32 errors of the scores 30 times larger too,
    # 2^-16 x 1200: 2^-5 of a weight (that is 2^-6 of its own and of the sum's)
    case = E.chunk_case(*lens, 8, 2, 128, 16, seed=21, q_mult=30.0)
    ref, tol = E.chunk_want(case)
    E.chunk_check(run(case), case, ref, 16 * tol)


@pytest.mark.parametrize("mods", [{}, dict(softcap=30.0)], ids=["plain", "capped"])
@pytest.mark.parametrize("most", [3, 30])
def test_many_short_sequences(mods, most):
    rng = np.random.default_rng(3)
    q = rng.integers(0, most, 1500)
    q[rng.random(1500) < 0.3] = 0
    ctx = q + rng.integers(0, 40, 1500)
    case = E.chunk_case(q.tolist(), ctx.tolist(), 4, 2, 64, 16, seed=14, **mods)
    E.chunk_check(run(case), case)


@pytest.mark.parametrize("mods", [{}, dict(softcap=30.0), dict(bias=True)], ids=["plain", "capped", "biased"])
@pytest.mark.parametrize("D", [64, 128])
def test_many_ragged_tails(D, mods):
    rng = np.random.default_rng(4)
    q = rng.integers(17, 40, 900)
    ctx = q + rng.choice([0, 30, 70, 140, 200], 900)
    ctx += ctx % 16 == 0
    case = E.chunk_case(q.tolist(), ctx.tolist(), 8, 2, D, 16, seed=24, **mods)
    E.chunk_check(run(case), case)


def test_many_pieces_per_row():
    for q, H_q, D, bs in (([1, 1], 8, 128, 16), ([2, 1], 8, 64, 32), ([40, 1], 8, 128, 16), ([1, 1], 16, 64, 32)):
        case = E.chunk_case(q, [6000 + q[0], 7001], H_q, 1, D, bs, seed=15)
        E.chunk_check(run(case, split_tokens=128), case)


@pytest.mark.parametrize("n", [1, 2, 40])
def test_a_sequence_of_a_hundred_thousand_tokens(n):
    case = E.chunk_case([n], [150_001], 1, 1, 64, 16, bias=True, seed=17)
    E.chunk_check(run(case), case)
    case = E.chunk_case([n], [150_001], 8, 1, 64, 16, window=3000, prefix=[5], seed=17)
    E.chunk_check(run(case), case)


def test_scales_of_the_whole_range():
    # groups' scales from 2^-9 to 448 in one row of keys and values, zero scales
    # and both zeros among the codes
    case = E.chunk_case([1, 2, 20], [300, 200, 90], 8, 2, 128, 16, seed=61, scaled=False)
    rng = np.random.default_rng(61)
    from oracle import formats as F
    for name, val in (("kc", "kval"), ("vc", "vval")):
        codes, sc = F.e2m1_unpack(case[name].numpy())
        bad = sc == 0x7F
        sc = np.where(bad, sc, rng.choice([0x00, 0x01, 0x07, 0x08, 0x20, 0x38, 0x50] + [0x7E] * (val == "vval"), sc.shape))
        case[name] = torch.from_numpy(F.e2m1_pack(codes, sc.astype(np.uint8)))
        case[val] = F.e2m1_values(F.e2m1_pack(codes, np.where(bad, 0, sc).astype(np.uint8)))
    ref, tol = E.chunk_want(case)
    E.chunk_check(run(case), case, ref, tol)


def test_shared_scales_and_row_strides():
    case = E.chunk_case(*FEW, 8, 2, 128, 16, seed=19)
    case["ks"], case["vs"] = case["ks"][:1].expand(8, 2).contiguous(), case["vs"][:1].expand(8, 2).contiguous()
    ref, tol = E.chunk_want(case)
    E.chunk_check(run(case), case, ref, tol)
    heads = dict(k_scale=case["ks"][0].contiguous().to(DEV), v_scale=case["vs"][0].contiguous().to(DEV))
    E.chunk_check(run(case, **heads), case, ref, tol)
    wide = torch.full((8, 5), float("nan"))
    wk, wv = wide.clone(), wide.clone()
    wk[:, :2], wv[:, :2] = case["ks"], case["vs"]
    E.chunk_check(run(case, k_scale=wk.to(DEV), v_scale=wv.to(DEV), scale_row_stride=5), case, ref, tol)


@pytest.mark.parametrize("lens", [SINGLE, RAGGED], ids=["single", "ragged"])
def test_two_calls_at_once_and_captured(lens):
    cases = [E.chunk_case(*lens, 8, 2, 128, 16, seed=51), E.chunk_case(*lens, 8, 2, 128, 16, softcap=20.0, seed=52)]
    args = [C.device_args(c, DEV) for c in cases]
    wants = [E.chunk_want(c) for c in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    outs = [[], []]
    for _ in range(5):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                outs[i].append(pkv.chunk_attention(*args[i][0], **dict(args[i][1], split_tokens=128 if i else 0)))
    torch.cuda.synchronize()
    assert pkv.device_error(DEV) == 0
    for c, w, os in zip(cases, wants, outs):
        for o in os:
            E.chunk_check(o, c, *w)
            assert torch.equal(o, os[0])
    g = torch.cuda.CUDAGraph()
    out, ws = torch.empty_like(args[0][0][0]), torch.empty(64 << 20, dtype=torch.uint8, device=DEV)
    with torch.cuda.graph(g):
        pkv.chunk_attention(*args[0][0], **dict(args[0][1], out=out, workspace=ws, split_tokens=128))
    g.replay()
    torch.cuda.synchronize()
    E.chunk_check(out, cases[0], *wants[0])
    args[0][0][0].copy_(cases[1]["q"])              # new queries through the captured pointers
    cases[0]["q"] = cases[1]["q"]
    g.replay()
    torch.cuda.synchronize()
    E.chunk_check(out, cases[0])


def test_a_far_block():
    # block ids past 2^19 at 4 KV heads: byte offsets beyond 2^31
    nb, bs, hkv, d = 600_000, 16, 4, 128
    kc = pkv.e2m1_cache(nb, hkv, bs, d, device=DEV)
    vc = pkv.e2m1_cache(nb, hkv, bs, d, device=DEV)
    for q in ([1, 1], [3, 40]):
        case = E.chunk_case(q, [500, 450], 8, hkv, d, bs, seed=8)
        far = nb - case["kc"].shape[0]
        kc[far:] = case["kc"].to(DEV)
        vc[far:] = case["vc"].to(DEV)
        args, kw = C.device_args(case, DEV)
        table = torch.where(args[3] >= 0, args[3] + far, args[3])
        out = pkv.chunk_attention(args[0], kc, vc, table, *args[4:], **kw)
        assert pkv.device_error(DEV) == 0
        E.chunk_check(out, case)


@pytest.mark.parametrize("q_lens", [[1, 1, 1], [2, 1, 2], [4, 40, 3]], ids=["single", "few", "ragged"])
def test_bad_values_on_the_device_are_recorded_and_skipped(q_lens):
    case = E.chunk_case(q_lens, [100, 200, 50], 8, 2, 128, 16, seed=2)
    args, kw = C.device_args(case, DEV)
    args = list(args)
    good = pkv.chunk_attention(*args, **kw)
    last = sum(q_lens[:2])
    bad_start = args[5].clone()
    bad_start[3] = 10 ** 6                        # the last sequence past the rows
    out = torch.full_like(good, 2.0)
    pkv.chunk_attention(*args[:5], bad_start, args[6], **dict(kw, out=out))
    assert pkv.device_error(DEV) == 3
    assert torch.equal(out[:last], good[:last]) and torch.all(out[last:] == 2.0)
    for bad in (case["kc"].shape[0], -1, 2 ** 31 - 1):  # a table entry outside the pool reads as zeros
        t = args[3].clone()
        t[0, 0] = bad
        pkv.chunk_attention(*args[:3], t, *args[4:], **kw)
        assert pkv.device_error(DEV) == 2
    ctx = args[4].clone()
    ctx[1] = 10 ** 6                              # a length beyond the bound is clamped
    pkv.chunk_attention(*args[:4], ctx, *args[5:], **kw)
    assert pkv.device_error(DEV) == 3
    E.chunk_check(pkv.chunk_attention(*args, **kw), case)


def test_refusals():
    case = E.chunk_case([4, 1], [40, 20], 8, 2, 128, 16, seed=2)
    args, kw = C.device_args(case, DEV)
    one = torch.ones((2, 2), device=DEV)
    for bad in (dict(k_scale=one, v_scale=None), dict(k_scale=one[:1], v_scale=one[:1]),
                dict(k_scale=one.double(), v_scale=one.double())):
        with pytest.raises((TypeError, ValueError)):
            pkv.chunk_attention(*args, **dict(kw, **bad))
    with pytest.raises(ValueError):               # 64-wide queries over 128-wide caches
        pkv.chunk_attention(args[0][:, :, :64].contiguous(), *args[1:], **kw)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("kind", ["e2m1", "e4m3", "bf16"])
def test_what_ran_before_does_not_matter(kind, D):
    # 7 query heads per KV head leave four rows of a tile of 256 without queries; what
    # an earlier call left there must not choose how scores are capped
    g = torch.Generator().manual_seed(9)
    n, hkv, bs = 700, 2, 16
    blocks = -(-n // bs)
    if kind == "e2m1":
        kc, vc = (E.pool(g, blocks, hkv, bs, D, loud=False).to(DEV) for _ in range(2))
    else:
        kc, vc = (torch.randn((blocks, hkv, bs, D), generator=g).to(DEV, torch.bfloat16) for _ in range(2))
    ones = None if kind == "bf16" else torch.ones(hkv, device=DEV)
    if kind == "e4m3":
        kc, vc = kc.to(torch.float8_e4m3fn), vc.to(torch.float8_e4m3fn)
    table = torch.arange(blocks, dtype=torch.int32, device=DEV)[None]
    ctx, starts = (torch.tensor(x, dtype=torch.int32, device=DEV) for x in ([n], [0, n]))
    q = torch.randn((n, 8 * hkv, D), generator=g).to(DEV, torch.bfloat16)

    def run(q):
        return pkv.chunk_attention(q, kc, vc, table, ctx, starts, D ** -0.5, max_q_len=n, max_context_len=n, softcap=30.0,
                                   k_scale=ones, v_scale=ones)

    outs = []
    for mult in (1e-3, 1e4):
        for _ in range(20):
            run(q * mult)                            # all 256 rows of every tile, on every SM
        outs.append(run(q[:, : 7 * hkv].contiguous()))
    assert pkv.device_error(DEV) == 0
    assert torch.equal(outs[0], outs[1])
