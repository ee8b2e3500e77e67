"""GPU parity of ragged chunk attention against the float64 oracle."""

import numpy as np
import pytest
import torch

import paged_kv_cache_222_gb300 as pkv

from . import chunk_support as C

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda", 0)


def run(case, **kw):
    args, kwargs = C.device_args(case, DEV)
    kwargs.update(kw)
    out = pkv.chunk_attention(*args, **kwargs)
    assert pkv.device_error(DEV) == 0
    return out


# (q_lens, ctxs): single tokens, lengths of one, chunks over a past, whole
# prompts, empty sequences and sequences without new tokens
SINGLE = ([1, 1, 1, 1, 1, 1], [1, 2, 17, 64, 65, 1000])
RAGGED = ([1, 5, 0, 33, 130, 64, 2], [1, 5, 40, 33, 300, 900, 257])
PROMPTS = ([1, 127, 128, 129, 300], [1, 127, 128, 129, 300])


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("H_q,H_kv,D,bs", [(8, 1, 128, 16), (6, 2, 64, 32), (4, 4, 128, 32), (7, 1, 64, 16),
                                           (16, 1, 128, 16), (5, 1, 128, 32)])
@pytest.mark.parametrize("lens", [SINGLE, RAGGED, PROMPTS], ids=["single", "ragged", "prompts"])
def test_plain_scores(lens, H_q, H_kv, D, bs, kv):
    case = C.make_case(*lens, H_q, H_kv, D, bs, kv, seed=H_q * 100 + D)
    C.check(run(case), case)


MODS = [dict(softcap=5.0), dict(softcap=30.0), dict(bias=True), dict(window=1), dict(window=100), dict(window=5000),
        dict(prefix=3), dict(prefix=10 ** 6), dict(window=40, prefix=20), dict(window=130, prefix=200, bias=True),
        dict(softcap=20.0, bias=True, window=77)]


def _with_prefix(mods, n):
    m = dict(mods)
    if "prefix" in m:  # another prefix for every sequence, none for the first
        m["prefix"] = [0] + [m["prefix"] + i for i in range(n - 1)]
    return m


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("mods", MODS, ids=[",".join(f"{k}={v}" for k, v in m.items()) for m in MODS])
@pytest.mark.parametrize("lens", [SINGLE, RAGGED], ids=["single", "ragged"])
@pytest.mark.parametrize("D,bs", [(64, 16), (128, 16), (128, 32)])
def test_modified_scores(lens, mods, kv, D, bs):
    case = C.make_case(*lens, 8, 2, D, bs, kv, seed=77, **_with_prefix(mods, len(lens[0])))
    C.check(run(case), case)


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("softcap", [1e-3, 0.5, 1e4, 1e7, 1e30])
@pytest.mark.parametrize("lens", [SINGLE, RAGGED], ids=["single", "ragged"])
def test_tiny_and_enormous_caps(lens, softcap, bias, kv):
    # a cap far above every score changes nothing, one far below levels them
    case = C.make_case(*lens, 8, 2, 128, 16, kv, softcap=softcap, bias=bias, seed=78)
    C.check(run(case), case)


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("split_tokens", [128, 256, 640])
@pytest.mark.parametrize("mods", [{}, dict(window=300), dict(window=200, prefix=129), dict(softcap=9.0, bias=True)],
                         ids=["plain", "window", "window+prefix", "cap+bias"])
@pytest.mark.parametrize("lens", [SINGLE, RAGGED], ids=["single", "ragged"])
def test_splits(lens, mods, split_tokens, kv):
    case = C.make_case(*lens, 8, 1, 128, 16, kv, seed=5, **_with_prefix(mods, len(lens[0])))
    C.check(run(case, split_tokens=split_tokens), case)


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("q_lens", [[1] * 4, [40, 3, 200, 1]], ids=["single", "ragged"])
def test_blocks_behind_the_window_may_be_gone(q_lens, kv):
    case = C.make_case(q_lens, [700, 333, 512, 650], 8, 2, 128, 16, kv, window=50, prefix=[0, 16, 10, 33], seed=9,
                       free_behind_window=True)
    assert (case["table"][0, :20] == -1).any()
    for st in (0, 128):
        C.check(run(case, split_tokens=st), case)


@pytest.mark.parametrize("q_lens", [[8, 8, 8], [200, 4, 130]], ids=["few", "many"])
def test_queries_before_position_zero_give_zeros(q_lens):
    # contexts shorter than the new tokens, down to none at all
    case = C.make_case(q_lens, [5, 0, 8], 8, 2, 128, 16, prefix=[3, 3, 3], seed=3)
    out = run(case)
    C.check(out, case)
    assert torch.all(out[: q_lens[0] - 5] == 0)
    assert torch.all(out[q_lens[0]:q_lens[0] + q_lens[1]] == 0)


@pytest.mark.parametrize("q_lens", [[1, 1], [150, 3]], ids=["few", "many"])
def test_rows_behind_the_last_sequence_stay(q_lens):
    case = C.make_case(q_lens, [300, 20], 8, 2, 128, 16, tail_rows=7, seed=4)
    out = torch.full_like(case["q"], 3.5, device=DEV)
    assert run(case, out=out) is out
    C.check(out, case)
    assert torch.all(out[sum(q_lens):] == 3.5)


def test_empty_calls():
    case = C.make_case([0, 0], [10, 0], 8, 2, 128, 16)
    assert run(case).shape == (0, 8, 128)
    case = C.make_case([], [], 8, 2, 128, 16, tail_rows=3)
    out = torch.full_like(case["q"], 1.25, device=DEV)
    args, kw = C.device_args(case, DEV)
    pkv.chunk_attention(*args[:3], torch.zeros((0, 1), dtype=torch.int32, device=DEV), *args[4:], **dict(kw, out=out))
    assert torch.all(out == 1.25)


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("lens", [SINGLE, RAGGED], ids=["single", "ragged"])
def test_large_and_peaked_scores(lens, kv):
    # queries 30 times larger: softmax rows dominated by single keys, running
    # maxima that grow by hundreds; scores sum 30 times larger products, so
    # their binary32 error, 2^-16 x 240, may reach 2^-8 of a weight
    case = C.make_case(*lens, 8, 2, 128, 16, kv, seed=21, q_mult=30.0)
    ref, tol = C.want(case)
    C.check(run(case), case, ref, 2 * tol)


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("softcap,q_mult,bias", [(5.0, 30.0, False), (50.0, 12.0, False), (50.0, 40.0, False),
                                                 (30.0, 12.0, True)])
@pytest.mark.parametrize("lens", [SINGLE, RAGGED], ids=["single", "ragged"])
def test_caps_that_bite(lens, softcap, q_mult, bias, D, kv):
    # scores from far below the cap to many times it.  A product is off by at
    # most D 2^-23 sum |q k| scale (about 2^-16 x 8 x q_mult), which the cap's slope, at
    # most 1, does not enlarge; the cap's own error is below 3e-6 of a score up to
    # 0.35 softcap and cap x 2^-22 above: 2^-8 of a weight in all
    case = C.make_case(*lens, 8, 2, D, 16, kv, softcap=softcap, bias=bias, seed=41, q_mult=q_mult)
    ref, tol = C.want(case)
    C.check(run(case), case, ref, 2 * tol)


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
@pytest.mark.parametrize("mods", [{}, dict(softcap=30.0)], ids=["plain", "capped"])
def test_many_short_sequences(mods, kv):
    # more sequences than one round of the search over their starts looks at,
    # many of them without new tokens, more row tiles than SMs
    rng = np.random.default_rng(3)
    q = rng.integers(0, 30, 1500)
    q[rng.random(1500) < 0.3] = 0
    ctx = q + rng.integers(0, 40, 1500)
    case = C.make_case(q.tolist(), ctx.tolist(), 4, 2, 64, 16, kv, seed=14, **mods)
    C.check(run(case), case)


@pytest.mark.parametrize("mods", [{}, dict(softcap=30.0), dict(bias=True)], ids=["plain", "capped", "biased"])
@pytest.mark.parametrize("D", [64, 128])
def test_many_ragged_tails(D, mods):
    # units of one to four key tiles in turn, all of them ending inside a block:
    # their loads run ahead of the products of the unit before
    rng = np.random.default_rng(4)
    q = rng.integers(17, 40, 900)
    ctx = q + rng.choice([0, 30, 70, 140, 200], 900)
    ctx += ctx % 16 == 0
    case = C.make_case(q.tolist(), ctx.tolist(), 8, 2, D, 16, seed=24, **mods)
    C.check(run(case), case)


@pytest.mark.parametrize("n", [40, 300])
def test_many_pieces_per_row(n):
    # 47 and more pieces of 128 tokens: the merges by whole CTAs and by warps
    case = C.make_case([n, 1], [6000 + n, 7001], 8, 1, 128, 16, seed=15)
    C.check(run(case, split_tokens=128), case)
    case = C.make_case([1, 1], [6000, 7001], 16, 1, 64, 32, "e4m3", seed=16)
    C.check(run(case, split_tokens=128), case)


@pytest.mark.parametrize("n", [1, 40])
def test_a_sequence_of_a_hundred_thousand_tokens(n):
    case = C.make_case([n], [150_001], 1, 1, 64, 16, bias=True, seed=17)
    C.check(run(case), case)
    case = C.make_case([n], [150_001], 1, 1, 64, 16, window=3000, prefix=[5], seed=17)
    C.check(run(case), case)


def test_two_calls_at_once_on_two_streams():
    cases = [C.make_case(*RAGGED, 8, 2, 128, 16, seed=51), C.make_case(*RAGGED, 8, 2, 128, 16, softcap=20.0, seed=52)]
    args = [C.device_args(c, DEV) for c in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    outs = [[], []]
    for _ in range(5):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                outs[i].append(pkv.chunk_attention(*args[i][0], **dict(args[i][1], split_tokens=128 if i else 0)))
    torch.cuda.synchronize()
    assert pkv.device_error(DEV) == 0
    for i, c in enumerate(cases):
        ref, tol = C.want(c)
        for o in outs[i]:
            C.check(o, c, ref, tol)


def test_default_bounds_are_the_tensors_own():
    case = C.make_case(*RAGGED, 8, 2, 128, 16, seed=53)
    args, kw = C.device_args(case, DEV)
    out = pkv.chunk_attention(*args)
    assert pkv.device_error(DEV) == 0
    C.check(out, case)


def test_refusals():
    case = C.make_case([4, 1], [40, 20], 8, 2, 128, 16, seed=2)
    args, kw = C.device_args(case, DEV)
    q, k, v, t, c, s, scale = args
    call = pkv.chunk_attention
    for bad, err in [
        ((q.float(), k, v, t, c, s, scale), TypeError), ((q[:, :, :64].contiguous(), k, v, t, c, s, scale), ValueError),
        ((q.transpose(0, 1), k, v, t, c, s, scale), ValueError), ((q, k, v[:-1], t, c, s, scale), ValueError),
        ((q, k, v, t.long(), c, s, scale), TypeError), ((q, k, v, t[:1], c, s, scale), ValueError),
        ((q, k, v, t, c[:1], s, scale), ValueError), ((q, k, v, t, c, s[:-1], scale), ValueError),
        ((q, k, v, t, c, s.cpu(), scale), ValueError), ((q, k, v, t, c, s, 0.0), pkv.PkvError),
        ((q[:, :7].contiguous(), k, v, t, c, s, scale), pkv.PkvError),
    ]:
        with pytest.raises(err):
            call(*bad, **kw)
    for bad, err in [(dict(out=torch.empty_like(q).float()), TypeError), (dict(out=q[:1]), ValueError),
                     (dict(slopes=torch.zeros(7, device=DEV)), ValueError),
                     (dict(prefix_lens=torch.zeros(3, dtype=torch.int32, device=DEV)), ValueError),
                     (dict(softcap=-1.0), pkv.PkvError), (dict(window=-1), pkv.PkvError),
                     (dict(max_context_len=10 ** 6), pkv.PkvError), (dict(split_tokens=100), pkv.PkvError),
                     (dict(k_scale=torch.ones(2, device=DEV)), ValueError),
                     (dict(split_tokens=128, max_context_len=48, workspace=torch.empty(0, dtype=torch.uint8, device=DEV)),
                      None)]:
        if err is None:
            call(*args, **dict(kw, **bad))  # one piece: no workspace needed
            continue
        with pytest.raises(err):
            call(*args, **dict(kw, **bad))
    with pytest.raises(pkv.PkvError):  # two pieces, too little workspace
        big = C.make_case([1], [400], 8, 2, 128, 16)
        a, kk = C.device_args(big, DEV)
        call(*a, **dict(kk, split_tokens=128, workspace=torch.empty(256, dtype=torch.uint8, device=DEV)))
    assert pkv.device_error(DEV) == 0


def test_a_long_sequence_and_far_blocks():
    # block ids past 2^17 at 8 KV heads: byte offsets beyond 2^32
    nb, bs, hkv, d = 140_000, 16, 8, 128
    kc = torch.zeros((nb, hkv, bs, d), dtype=torch.bfloat16, device=DEV)
    vc = torch.zeros_like(kc)
    case = C.make_case([3, 40], [500, 450], 16, hkv, d, bs, seed=8)
    far = nb - case["kc"].shape[0]
    kc[far:] = case["kc"].to(DEV)
    vc[far:] = case["vc"].to(DEV)
    args, kw = C.device_args(case, DEV)
    table = torch.where(args[3] >= 0, args[3] + far, args[3])
    out = pkv.chunk_attention(args[0], kc, vc, table, *args[4:], **kw)
    assert pkv.device_error(DEV) == 0
    C.check(out, case)


def test_single_tokens_agree_with_decode_attention():
    case = C.make_case(*SINGLE, 8, 2, 128, 16, seed=6)
    args, kw = C.device_args(case, DEV)
    dec = pkv.decode_attention(args[0], *args[1:5], case["scale"], max_context_len=case["max_ctx"])
    _, tol = C.want(case)
    err = (run(case).double() - dec.double()).abs().cpu().numpy()
    assert (err <= tol + 2e-3 * 2.0 ** -3).all()


@pytest.mark.parametrize("lens", [SINGLE, RAGGED], ids=["single", "ragged"])
def test_captured_graphs_with_workspaces_of_their_own(lens):
    cases = [C.make_case(*lens, 8, 2, 128, 16, seed=s) for s in (31, 32)]
    refs = [C.want(c) for c in cases]
    runs = []
    for c in cases:
        args, kw = C.device_args(c, DEV)
        out = torch.empty_like(args[0])
        ws = torch.empty(64 << 20, dtype=torch.uint8, device=DEV)
        kw.update(out=out, workspace=ws, split_tokens=128)
        pkv.chunk_attention(*args, **kw)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            pkv.chunk_attention(*args, **kw)
        runs.append((g, out, args, kw))  # a graph's inputs and workspace live as long as it is replayed
    streams = [torch.cuda.Stream() for _ in runs]
    for _, out, _, _ in runs:
        out.zero_()
    torch.cuda.synchronize()
    for _ in range(3):
        for (g, _, _, _), s in zip(runs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for (_, out, _, _), c, (ref, tol) in zip(runs, cases, refs):
        C.check(out, c, ref, tol)
    # new inputs through the captured pointers
    g, out, args, _ = runs[0]
    args[0].copy_(cases[1]["q"])
    cases[0]["q"] = cases[1]["q"]
    g.replay()
    torch.cuda.synchronize()
    C.check(out, cases[0])


def test_two_calls_are_bit_equal():
    case = C.make_case(*RAGGED, 8, 2, 128, 16, softcap=20.0, seed=12)
    for st in (0, 128):
        assert torch.equal(run(case, split_tokens=st), run(case, split_tokens=st))


def test_bad_values_on_the_device_are_recorded_and_skipped():
    case = C.make_case([4, 40, 3], [100, 200, 50], 8, 2, 128, 16, seed=2)
    args, kw = C.device_args(case, DEV)
    args = list(args)
    good = pkv.chunk_attention(*args, **kw)
    bad_start = args[5].clone()
    bad_start[3] = 10 ** 6                        # the last sequence past the rows
    out = torch.full_like(good, 2.0)
    pkv.chunk_attention(*args[:5], bad_start, args[6], **dict(kw, out=out))
    assert pkv.device_error(DEV) == 3
    assert torch.equal(out[:44], good[:44]) and torch.all(out[44:] == 2.0)
    # a table entry outside the pool reads as zeros
    t = args[3].clone()
    t[0, 0] = case["kc"].shape[0]
    pkv.chunk_attention(*args[:3], t, *args[4:], **kw)
    assert pkv.device_error(DEV) == 2
    # a length beyond the bound is clamped
    ctx = args[4].clone()
    ctx[1] = 10 ** 6
    pkv.chunk_attention(*args[:4], ctx, *args[5:], **kw)
    assert pkv.device_error(DEV) == 3
    # longer than max_q_len: skipped
    out.fill_(2.0)
    pkv.chunk_attention(*args, **dict(kw, max_q_len=20, out=out))
    assert pkv.device_error(DEV) == 3
    assert torch.all(out[4:44] == 2.0)
    C.check(torch.cat([out[:4], good[4:44], out[44:]]), case)
