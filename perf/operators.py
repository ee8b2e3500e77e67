"""Measured cases of the prompt-side operators of the paged cache.

Three operators make up what a serving step does around the cache when whole
chunks of new tokens arrive, next to single tokens:

  chunk    chunk_attention: every sequence's new tokens (one, or thousands)
           attend its paged keys and values causally, with the scores as the
           model defines them: capped by a tanh, biased by distance, limited
           to a window, opened for a prefix; caches in bf16 or E4M3
  rotary   rotary_append: new queries and keys are turned by their rotary
           angles, the queries returned, keys and values written to their slots
  compact  compact_tokens: the kept tokens of every sequence move to the front
           of its blocks (after eviction, or after a draft was judged)

`listed` names the cases, `draw` gives more of the same ranges.  `run` takes
the state of `prepare` through one operator: in plain torch operations where
`own` is false, through the package's call where it is true.  `exact` is the
definition in 64 bits.
"""

import math
import random

import numpy as np
import torch

own = False

DEV = "cuda"


# ---------------------------------------------------------------- cases

def listed():
    return [
        # the second half of two long prompts: chunked prefill of the 70B-class
        # attention geometry, 4096 new tokens over 4096 cached ones
        chunk("chunk 4096 of 8192", B=2, q=(4096, 4096), past=(4096, 4096)),
        # chunks of very different lengths in one call, some of one token (a
        # decode step riding along), over an E4M3 cache with 32-token blocks
        chunk("ragged chunks e4m3", B=12, q=(1, 512), past=(0, 3584), bs=32, kv="e4m3"),
        # a whole prompt through a layer with a sliding window and capped scores
        chunk("prompt windowed capped", B=1, q=(8191, 8191), past=(0, 0), H_q=32, window=1024, softcap=50.0),
        # whole prompts of odd lengths with distance bias and a prefix seen from
        # both sides, seven query heads per key head, 64-wide heads
        chunk("prompts biased prefix d64", B=5, q=(301, 1777), past=(0, 0), H_q=28, H_kv=4, D=64, bias=True,
              prefix=(0, 700)),
        # a decode step of 64 sequences with capped scores
        chunk("decode capped", B=64, q=(1, 1), past=(511, 8191), softcap=30.0),
        # a decode step of 256 sequences over an E4M3 cache, a window behind
        # sixteen tokens that stay visible
        chunk("decode windowed e4m3", B=256, q=(1, 1), past=(2047, 4095), kv="e4m3", window=1024, prefix=(16, 16)),
        # the smallest call: one new token of one short sequence
        chunk("one token", B=1, q=(1, 1), past=(99, 99), H_q=4, H_kv=1, D=64),
        # a decode step's 64 new tokens, three of them padding
        rotary("rotary decode step", N=64, far=131072, pad=3),
        # a prompt of 8192 tokens
        rotary("rotary prompt", N=8192, far=8192, run=True),
        # an odd number of new tokens far into a scaled context, interleaved
        # pairs over half of the head, float32 inputs quantised to E4M3
        rotary("rotary partial scaled e4m3", N=1777, far=1 << 20, H_q=32, D=128, rd=64, interleaved=True, factor=8.0,
               src="f32", kv="e4m3"),
        # half of the tokens of 32 long sequences are evicted
        compact("evict half of 4096", B=32, length=(4096, 4096), keep=0.5, first=4),
        # eight of the last sixteen draft tokens of each of 64 sequences stay
        compact("accepted drafts", B=64, length=(500, 2048), draft=16, accept=8, kv="e4m3"),
    ]


def chunk(name=None, B=1, q=(1, 1), past=(0, 0), H_q=64, H_kv=8, D=128, bs=16, kv="bf16", softcap=0.0, window=0,
          bias=False, prefix=(0, 0), shape=1):
    c = dict(op="chunk", B=B, q_min=q[0], q_max=q[1], past_min=past[0], past_max=past[1], H_q=H_q, H_kv=H_kv, D=D,
             bs=bs, kv=kv, softcap=float(softcap), window=window, bias=bias, prefix_min=prefix[0],
             prefix_max=prefix[1], shape=shape)
    return dict(c, name=name) if name else c


def rotary(name=None, N=1, far=4096, pad=0, run=False, H_q=64, H_kv=8, D=128, rd=None, bs=16, interleaved=False,
           factor=1.0, src="bf16", kv="bf16"):
    c = dict(op="rotary", N=N, far=far, pad=pad, run=run, H_q=H_q, H_kv=H_kv, D=D, rd=rd or D, bs=bs,
             interleaved=interleaved, factor=float(factor), src=src, kv=kv)
    return dict(c, name=name) if name else c


def compact(name=None, B=1, length=(16, 16), keep=0.0, first=0, draft=0, accept=0, H_kv=8, D=128, bs=16, kv="bf16",
            shape=1):
    c = dict(op="compact", B=B, len_min=length[0], len_max=length[1], keep=float(keep), first=first, draft=draft,
             accept=accept, H_kv=H_kv, D=D, bs=bs, kv=kv, shape=shape)
    return dict(c, name=name) if name else c


def _log(rng, lo, hi):
    """A whole number of [lo, hi], spread over its logarithm."""
    return min(hi, max(lo, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def draw(rng):
    op = rng.choice(["chunk", "chunk", "chunk", "rotary", "compact"])
    D, bs, kv = rng.choice([64, 128, 128]), rng.choice([16, 32]), rng.choice(["bf16", "bf16", "e4m3"])
    H_kv = rng.choice([1, 2, 4, 8])
    if op == "rotary":
        G = rng.choice([1, 2, 3, 4, 5, 8])
        return rotary(N=_log(rng, 1, 8192), far=_log(rng, 8192, 1 << 20), pad=rng.choice([0, 0, 1]),
                      run=rng.random() < 0.5, H_q=H_kv * G, H_kv=H_kv, D=D, rd=rng.choice([D, D, D // 2, 16]), bs=bs,
                      interleaved=rng.random() < 0.5, factor=rng.choice([1.0, 4.0, 32.0]),
                      src=rng.choice(["bf16", "f32"]), kv=kv)
    if op == "compact":
        B = _log(rng, 1, 64)
        if rng.random() < 0.5:
            n = _log(rng, 2, 32)
            hi = _log(rng, 64, 4096)
            return compact(B=B, length=(hi // 2, hi), draft=n, accept=rng.randint(1, n), H_kv=H_kv, D=D, bs=bs, kv=kv,
                           shape=rng.randrange(1 << 20))
        hi = _log(rng, 64, 4096)
        return compact(B=B, length=(hi // 2, hi), keep=rng.uniform(0.1, 0.9), first=rng.choice([0, 4]), H_kv=H_kv, D=D,
                       bs=bs, kv=kv, shape=rng.randrange(1 << 20))
    G = rng.choice([1, 2, 3, 4, 5, 6, 7, 8, 12, 16])
    H_q = H_kv * G
    kind = rng.choice(["decode", "chunks", "chunks", "prompts"])
    if kind == "decode":
        B = _log(rng, 1, 128)
        hi = _log(rng, 64, 8191)
        q, past = (1, 1), (hi // 4, hi)
    else:
        B = _log(rng, 1, 16)
        room = 2.0e9 / (B * H_q)                      # padded scores of the plain form, in elements
        hi = _log(rng, 2, max(2, min(4096, int(math.sqrt(room)))))
        q = (max(1, hi // 8), hi)
        past = (0, 0) if kind == "prompts" else (0, _log(rng, 1, max(1, min(12288, int(room / hi) - hi))))
    return chunk(B=B, q=q, past=past, H_q=H_q, H_kv=H_kv, D=D, bs=bs, kv=kv,
                 softcap=rng.choice([0.0, 0.0, 30.0, 50.0]), window=rng.choice([0, 0, 0, _log(rng, 16, 2048)]),
                 bias=rng.random() < 0.25, prefix=rng.choice([(0, 0), (0, 0), (1, 300)]), shape=rng.randrange(1 << 20))


def _chunk_lens(c):
    """(q_len, context, prefix) of every sequence, from the case alone."""
    r = random.Random(c["shape"])
    q = [r.randint(c["q_min"], c["q_max"]) for _ in range(c["B"])]
    ctx = [n + r.randint(c["past_min"], c["past_max"]) for n in q]
    return q, ctx, [r.randint(c["prefix_min"], c["prefix_max"]) for _ in range(c["B"])]


def _compact_lens(c):
    """(length, first destination, kept) of every sequence, from the case alone."""
    r = random.Random(c["shape"])
    length = [r.randint(max(c["len_min"], c["draft"], 1), max(c["len_max"], c["draft"], 1)) for _ in range(c["B"])]
    if c["draft"]:
        return length, [n - c["draft"] for n in length], [c["accept"]] * c["B"]
    return length, [min(c["first"], n) for n in length], [int((n - min(c["first"], n)) * c["keep"]) for n in length]


# ---------------------------------------------------------------- inputs

def prepare(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(int(seed))
    return {"chunk": _prepare_chunk, "rotary": _prepare_rotary, "compact": _prepare_compact}[case["op"]](case, gen)


def _randn(gen, *shape):
    return torch.randn(shape, generator=gen, device=DEV)


def _pool(gen, c, blocks):
    """K and V pools; E4M3 codes of values up to about 448 / 64 scales."""
    shape = (blocks, c["H_kv"], c["bs"], c["D"])
    if c["kv"] == "bf16":
        return _randn(gen, *shape).bfloat16(), _randn(gen, *shape).bfloat16()
    return tuple((_randn(gen, *shape) * 64.0).clamp(-448.0, 448.0).to(torch.float8_e4m3fn) for _ in range(2))


def _tables(gen, lens, bs):
    """Block tables over a shuffled pool (-1 past each sequence), and the pool's size."""
    need = torch.tensor([-(-n // bs) for n in lens], device=DEV)
    total, most = int(need.sum()) + 3, max(1, int(need.max()))
    order = torch.randperm(total, generator=gen, device=DEV)
    first = torch.cumsum(need, 0) - need
    j = torch.arange(most, device=DEV)
    at = (first[:, None] + j).clamp(max=total - 1)
    return torch.where(j < need[:, None], order[at], -1).to(torch.int32), total


def _scales(gen, *shape):
    return (0.5 + torch.rand(shape, generator=gen, device=DEV)) / 64.0


def _prepare_chunk(c, gen):
    q_len, ctx, prefix = _chunk_lens(c)
    tables, blocks = _tables(gen, ctx, c["bs"])
    k, v = _pool(gen, c, blocks)
    starts = [0]
    for n in q_len:
        starts.append(starts[-1] + n)
    s = {"case": c, "k": k, "v": v, "tables": tables, "max_q": max(q_len), "max_ctx": max(ctx),
         "q": _randn(gen, starts[-1], c["H_q"], c["D"]).bfloat16(),
         "starts": torch.tensor(starts, dtype=torch.int32, device=DEV),
         "ctx": torch.tensor(ctx, dtype=torch.int32, device=DEV), "scale": c["D"] ** -0.5,
         "slopes": None, "prefix": None, "ks": None, "vs": None}
    if c["bias"]:
        s["slopes"] = torch.exp2(-8.0 * torch.arange(1, c["H_q"] + 1, device=DEV) / c["H_q"]).float()
    if c["prefix_max"]:
        s["prefix"] = torch.tensor(prefix, dtype=torch.int32, device=DEV)
    if c["kv"] == "e4m3":
        s["ks"], s["vs"] = _scales(gen, c["B"], c["H_kv"]), _scales(gen, c["B"], c["H_kv"])
    return s


def _inv_freq(c):
    """Rotary frequencies in 64 bits: base 10000, and for scaled contexts each
    frequency divided by the factor as far as its turns over the original
    context stay below 32 (wholly below one turn)."""
    i = torch.arange(0, c["rd"], 2, dtype=torch.float64)
    f = 10000.0 ** (-i / c["rd"])
    if c["factor"] > 1.0:
        turns = 8192.0 * f / (2.0 * math.pi)
        keep = ((turns - 1.0) / 31.0).clamp(0.0, 1.0)
        f = f * (keep + (1.0 - keep) / c["factor"])
    return f.to(DEV)


def _prepare_rotary(c, gen):
    N, bs, dt = c["N"], c["bs"], torch.bfloat16 if c["src"] == "bf16" else torch.float32
    blocks = -(-N // bs) + 2
    k_cache, v_cache = _pool(gen, c, blocks)
    if c["run"]:                                     # a prompt: consecutive positions and slots in shuffled blocks
        pos = torch.arange(N, device=DEV) + (c["far"] - N if c["far"] > N else 0)
        order = torch.randperm(blocks, generator=gen, device=DEV)
        at = torch.arange(N, device=DEV)
        slots = order[at // bs] * bs + at % bs
    else:                                            # one token of each of N sequences
        pos = torch.randint(0, c["far"], (N,), generator=gen, device=DEV)
        slots = torch.randperm(blocks * bs, generator=gen, device=DEV)[:N]
    if c["pad"]:
        slots = torch.where(torch.arange(N, device=DEV) < N - c["pad"], slots, -1)
    s = {"case": c, "q": _randn(gen, N, c["H_q"], c["D"]).to(dt), "kn": _randn(gen, N, c["H_kv"], c["D"]).to(dt),
         "vn": _randn(gen, N, c["H_kv"], c["D"]).to(dt), "pos": pos, "slots": slots, "f": _inv_freq(c),
         "mag": 1.0 + 0.1 * math.log(c["factor"]), "k": k_cache, "v": v_cache, "ks": None, "vs": None}
    if c["kv"] == "e4m3":
        s["ks"], s["vs"] = _scales(gen, N, c["H_kv"]), _scales(gen, N, c["H_kv"])
    return s


def _prepare_compact(c, gen):
    length, first, kept = _compact_lens(c)
    tables, blocks = _tables(gen, length, c["bs"])
    k, v = _pool(gen, c, blocks)
    # the kept positions of each sequence: a random choice, in order
    starts = [0]
    for n in kept:
        starts.append(starts[-1] + n)
    most = max(max(n - f for n, f in zip(length, first)), 1)
    j = torch.arange(most, device=DEV)
    room = torch.tensor([n - f for n, f in zip(length, first)], device=DEV)
    key = torch.rand((c["B"], most), generator=gen, device=DEV)
    key = torch.where(j < room[:, None], key, 2.0)
    rank = key.argsort(1).argsort(1)
    chosen = rank < torch.tensor(kept, device=DEV)[:, None]
    b, p = chosen.nonzero(as_tuple=True)
    first = torch.tensor(first, device=DEV)
    return {"case": c, "k": k, "v": v, "tables": tables, "keep": (p + first[b]).to(torch.int32),
            "starts": torch.tensor(starts, dtype=torch.int32, device=DEV), "first": first.to(torch.int32),
            "most": max(kept)}


# ---------------------------------------------------------------- one pass

def run(state):
    return {"chunk": _run_chunk, "rotary": _run_rotary, "compact": _run_compact}[state["case"]["op"]](state)


def _rows_of(tables, cache):
    """Every token row a table addresses, as float32 [B, H_kv, MB * bs, D]."""
    B, MB = tables.shape
    _, H, bs, D = cache.shape
    # E4M3 pools are picked as the bytes they are
    raw = cache.view(torch.uint8) if cache.dtype == torch.float8_e4m3fn else cache
    x = raw[tables.long().clamp(min=0)].view(cache.dtype).float()
    return x.permute(0, 2, 1, 3, 4).reshape(B, H, MB * bs, D)


def _run_chunk(s):
    c = s["case"]
    if own:
        import paged_kv_cache_222_gb300 as pkv
        return pkv.chunk_attention(s["q"], s["k"], s["v"], s["tables"], s["ctx"], s["starts"], s["scale"],
                                   max_q_len=s["max_q"], max_context_len=s["max_ctx"], k_scale=s["ks"],
                                   v_scale=s["vs"], softcap=c["softcap"], window=c["window"], slopes=s["slopes"],
                                   prefix_lens=s["prefix"])
    B, H_q, H, D = c["B"], c["H_q"], c["H_kv"], c["D"]
    G, L = H_q // H, s["max_q"]
    starts, ctx = s["starts"].long(), s["ctx"].long()
    n = starts[1:] - starts[:-1]
    K, V = _rows_of(s["tables"], s["k"]), _rows_of(s["tables"], s["v"])
    if s["ks"] is not None:
        K, V = K * s["ks"][:, :, None, None], V * s["vs"][:, :, None, None]
    i = torch.arange(L, device=DEV)
    at = (starts[:-1, None] + i).clamp(max=s["q"].shape[0] - 1)
    q = s["q"].float()[at].view(B, L, H, G, D).permute(0, 2, 3, 1, 4).reshape(B, H, G * L, D)
    x = (q @ K.transpose(2, 3)).view(B, H, G, L, -1) * s["scale"]
    if c["softcap"]:
        x = c["softcap"] * torch.tanh(x / c["softcap"])
    t = torch.arange(K.shape[2], device=DEV)
    pos = (ctx - n)[:, None] + i                                            # [B, L]
    away = t - pos[:, :, None]                                              # [B, L, T]
    if s["slopes"] is not None:
        x = x + s["slopes"].view(1, H, G, 1, 1) * away[:, None, None]
    see = away <= 0
    if c["window"]:
        see = see & (away > -c["window"])
    if s["prefix"] is not None:
        see = see | (t < s["prefix"][:, None, None])
    see = see & (t < ctx[:, None, None]) & (pos >= 0)[:, :, None]
    x = torch.where(see[:, None, None], x, -math.inf)
    m = x.amax(-1, keepdim=True).clamp(min=-3e38)
    p = torch.exp(x - m)
    total = p.sum(-1, keepdim=True)
    V = torch.where((t < ctx[:, None])[:, None, :, None], V, 0.0)
    o = (p.view(B, H, G * L, -1) @ V).view(B, H, G, L, D) / total.clamp(min=1e-38)
    o = o.permute(0, 3, 1, 2, 4).reshape(B, L, H_q, D)
    return o[i < n[:, None]].bfloat16()


def _turned(x, cos, sin, rd, interleaved):
    a = x[..., :rd]
    if interleaved:
        u, w = a[..., 0::2], a[..., 1::2]
        y = torch.stack((u * cos - w * sin, w * cos + u * sin), -1).flatten(-2)
    else:
        u, w = a[..., :rd // 2], a[..., rd // 2:]
        y = torch.cat((u * cos - w * sin, w * cos + u * sin), -1)
    return torch.cat((y, x[..., rd:]), -1)


def _run_rotary(s):
    c = s["case"]
    if own:
        import paged_kv_cache_222_gb300 as pkv
        q = pkv.rotary_append(s["q"], s["kn"], s["vn"], s["pos"], s["f"], s["slots"], s["k"], s["v"], k_scale=s["ks"],
                              v_scale=s["vs"], magnitude=s["mag"], interleaved=c["interleaved"])
        return q, s["k"], s["v"]
    angle = s["pos"].double()[:, None] * s["f"]
    cos, sin = (f(angle).float()[:, None] * s["mag"] for f in (torch.cos, torch.sin))
    q = _turned(s["q"].float(), cos, sin, c["rd"], c["interleaved"]).bfloat16()
    k, v = _turned(s["kn"].float(), cos, sin, c["rd"], c["interleaved"]), s["vn"].float()
    if s["ks"] is not None:
        k = (k / s["ks"][:, :, None]).clamp(-448.0, 448.0)
        v = (v / s["vs"][:, :, None]).clamp(-448.0, 448.0)
    live = s["slots"] >= 0
    slot = s["slots"][live]
    blk, off = slot // c["bs"], slot % c["bs"]
    for cache, rows in ((s["k"], k), (s["v"], v)):
        rows = rows[live].to(cache.dtype)
        if cache.dtype == torch.float8_e4m3fn:
            cache, rows = cache.view(torch.uint8), rows.view(torch.uint8)
        cache[blk, :, off] = rows
    return q, s["k"], s["v"]


def _run_compact(s):
    if own:
        import paged_kv_cache_222_gb300 as pkv
        pkv.compact_tokens(s["k"], s["v"], s["tables"], s["keep"], s["starts"], dst_start=s["first"],
                           max_keep=s["most"])
        return s["k"], s["v"]
    bs = s["k"].shape[2]
    starts, keep = s["starts"].long(), s["keep"].long()
    e = torch.arange(keep.numel(), device=DEV)
    b = torch.searchsorted(starts, e, right=True) - 1
    dst = s["first"].long()[b] + e - starts[b]
    table = s["tables"].long()
    from_blk, from_off = table[b, keep // bs], keep % bs
    to_blk, to_off = table[b, dst // bs], dst % bs
    for cache in (s["k"], s["v"]):
        raw = cache.view(torch.uint8) if cache.dtype == torch.float8_e4m3fn else cache
        raw[to_blk, :, to_off] = raw[from_blk, :, from_off]
    return s["k"], s["v"]


# ---------------------------------------------------------------- what a pass cannot do without

def work(case):
    return {"chunk": _work_chunk, "rotary": _work_rotary, "compact": _work_compact}[case["op"]](case)


def _work_chunk(c):
    """Every query read and output written once, every key and value that some
    query sees read once; two products per query head and visible pair."""
    size = 2 if c["kv"] == "bf16" else 1
    pairs = seen = rows = 0
    for n, ctx, prefix in zip(*_chunk_lens(c)):
        pos = np.arange(ctx - n, ctx, dtype=np.int64)
        lo = np.maximum(0, pos - c["window"] + 1) if c["window"] else np.zeros_like(pos)
        p = min(prefix, ctx)
        both = np.maximum(0, np.minimum(pos + 1, p) - lo)                 # in the window and in the prefix
        pairs += int((pos + 1 - lo + p - both).sum())
        seen += min(ctx, p + max(0, ctx - max(p, int(lo[0]))))
        rows += n
    return {"bytes": 4 * rows * c["H_q"] * c["D"] + 2 * seen * c["H_kv"] * c["D"] * size,
            "flops": 4 * pairs * c["H_q"] * c["D"]}


def _work_rotary(c):
    src, dst = (2 if c["src"] == "bf16" else 4), (2 if c["kv"] == "bf16" else 1)
    live = c["N"] - c["pad"]
    return {"bytes": c["N"] * c["H_q"] * c["D"] * (src + 2) + 2 * live * c["H_kv"] * c["D"] * (src + dst),
            "flops": 3 * (c["N"] * c["H_q"] + live * c["H_kv"]) * c["rd"]}


def _work_compact(c):
    size = 2 if c["kv"] == "bf16" else 1
    return {"bytes": 4 * sum(_compact_lens(c)[2]) * c["H_kv"] * c["D"] * size, "flops": 0}


# ---------------------------------------------------------------- the definition in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    return {"chunk": _exact_chunk, "rotary": _exact_rotary, "compact": _exact_compact}[case["op"]](s)


def _exact_chunk(s):
    """Sequence by sequence, head by head: softmax over the visible keys."""
    c = s["case"]
    G, bs = c["H_q"] // c["H_kv"], c["bs"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEV)
    starts, ctxs = s["starts"].tolist(), s["ctx"].tolist()
    prefix = s["prefix"].tolist() if s["prefix"] is not None else [0] * c["B"]
    for b, ctx in enumerate(ctxs):
        n = starts[b + 1] - starts[b]
        ids = s["tables"][b, :-(-ctx // bs)].long()
        key = torch.arange(ctx, device=DEV)
        pos = torch.arange(ctx - n, ctx, device=DEV)
        d = pos[:, None] - key[None, :]                                    # how far back a key lies
        hidden = (d < 0) if not c["window"] else (d < 0) | (d >= c["window"])
        hidden &= (key >= prefix[b])[None, :]
        for h in range(c["H_kv"]):
            K, V = (torch.cat([x[j, h] for j in ids.tolist()]).double()[:ctx] for x in (s["k"], s["v"]))
            for g in range(h * G, (h + 1) * G):
                z = torch.einsum("id,td->it", s["q"][starts[b]:starts[b + 1], g].double(), K) * s["scale"]
                if s["ks"] is not None:
                    z *= s["ks"][b, h].double()
                if c["softcap"]:
                    z = torch.tanh(z / c["softcap"]) * c["softcap"]
                if s["slopes"] is not None:
                    z -= s["slopes"][g].double() * d
                w = torch.softmax(z.masked_fill(hidden, -math.inf), dim=1)
                o = torch.einsum("it,td->id", w, V)
                out[starts[b]:starts[b + 1], g] = o if s["vs"] is None else o * s["vs"][b, h].double()
    return out


def _exact_rotary(s):
    """Each pair as a complex number, times magnitude * e^(i angle)."""
    c = s["case"]
    rd, half = c["rd"], c["rd"] // 2
    angle = s["pos"].double()[:, None] * s["f"].double()[None, :]
    turn = torch.polar(torch.full_like(angle, s["mag"]), angle)[:, None]
    first = torch.arange(half, device=DEV) * 2 if c["interleaved"] else torch.arange(half, device=DEV)
    second = first + 1 if c["interleaved"] else first + half

    def turned(x):
        y = x.double().clone()
        z = torch.complex(y[..., first], y[..., second]) * turn
        y[..., first], y[..., second] = z.real, z.imag
        return y

    caches = []
    for cache, rows, scale in ((s["k"], turned(s["kn"]), s["ks"]), (s["v"], s["vn"].double(), s["vs"])):
        out = cache.double()
        if scale is not None:
            rows = (rows / scale.double()[:, :, None]).clamp(-448.0, 448.0)
        flat = out.permute(0, 2, 1, 3).reshape(-1, c["H_kv"], c["D"])
        live = s["slots"] >= 0
        flat[s["slots"][live]] = rows[live]
        caches.append(flat.view(out.shape[0], c["bs"], c["H_kv"], c["D"]).permute(0, 2, 1, 3).contiguous())
    return turned(s["q"]), caches[0], caches[1]


def _exact_compact(s):
    """Sequence by sequence, from a copy of what the pool held."""
    bs = s["case"]["bs"]
    starts, first = s["starts"].tolist(), s["first"].tolist()
    outs = []
    for cache in (s["k"], s["v"]):
        old, new = cache.double(), cache.double()
        for b in range(len(first)):
            src = s["keep"][starts[b]:starts[b + 1]].long()
            dst = first[b] + torch.arange(src.numel(), device=DEV)
            t = s["tables"][b].long()
            new[t[dst // bs], :, dst % bs] = old[t[src // bs], :, src % bs]
        outs.append(new)
    return tuple(outs)
