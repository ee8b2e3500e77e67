"""Measured cases of the operators around a 4-bit paged cache.

What a serving step does between the model's projections and its output, with
no number read back to the host, over caches of four and a half bits per value:

  tables   extend_tables / truncate_tables: every request's new tokens get
           blocks from a free list on the GPU, their slots, positions and the
           step's ragged offsets; tokens that leave give their blocks back
  rotary   rotary_append with several axes: every pair of a head is turned by
           the position along one axis (time, height, width)
  store    append and read_tokens over an E2M1 cache: new keys and values
           become 4-bit floating-point codes with an 8-bit scale for every 16
           of them, and the pool's tokens are read back as values
  attend   chunk_attention over an E2M1 cache: single tokens, chunks, prompts

An E2M1 cache is uint8 [blocks, heads, block_size, D / 2 + D / 16]; the bytes
of one block and head are block_size rows of D / 2 code bytes (element 2 i in
the low half of byte i) and then block_size rows of D / 16 scale bytes (E4M3).

`listed` names the cases, `draw` gives more of the same ranges.  `run` takes
the state of `prepare` through one operator: in plain torch operations where
`own` is false, through the package's calls where it is true.  `exact` is the
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
        # a decode step of 256 requests: one new token each, a new block for
        # some sixteenth of them
        tables("tables decode step", B=256, past=(1, 8191), new=(1, 1)),
        # a step that admits 96 whole prompts beside 928 decoding requests
        tables("tables prompts admitted", B=1024, past=(0, 4095), new=(1, 1), prompts=96, prompt=(17, 2600), pad=61,
               bs=32),
        # 64 finished requests give all of their blocks back
        tables("tables requests finished", B=64, past=(1, 32768), back=True),
        # a prompt of text, images and video of 8192 tokens, three axes in turn
        rotary("rotary axes prompt", N=8192, cuts=(16, 24, 24), span=2048),
        # a decode step's 61 tokens, axes interleaved pair by pair, E4M3 cache
        rotary("rotary axes decode", N=61, cuts=(24, 20, 20), mixed=True, span=32768, kv="e4m3", pad=3),
        # a prompt's keys and values quantised, the pool read back
        store("store prompt", N=8192, pool=8192),
        # a decode step's float32 rows of an odd number of heads, some padding
        store("store few f32", N=45, pool=96, H_kv=3, D=64, bs=32, src="f32", scaled=True, pad=4),
        # a decode step of 64 sequences
        attend("decode e2m1", B=64, q=(1, 1), past=(511, 8191)),
        # a decode step of 8 sequences of 131,072 tokens
        attend("decode long e2m1", B=8, q=(1, 1), past=(131071, 131071), scaled=False),
        # chunks of very different lengths in one call, single tokens among them
        attend("chunks e2m1", B=12, q=(1, 512), past=(0, 3584), bs=32),
        # whole prompts with capped scores, seven query heads per key head
        attend("prompts capped e2m1 d64", B=5, q=(301, 1777), past=(0, 0), H_q=28, H_kv=4, D=64, softcap=30.0),
        # the smallest call: one new token of one short sequence
        attend("one token e2m1", B=1, q=(1, 1), past=(99, 99), H_q=4, H_kv=1, D=64),
    ]


def tables(name=None, B=1, past=(0, 0), new=(1, 1), prompts=0, prompt=(1, 1), pad=0, bs=16, back=False, shape=1):
    c = dict(op="tables", B=B, past_min=past[0], past_max=past[1], new_min=new[0], new_max=new[1], prompts=prompts,
             prompt_min=prompt[0], prompt_max=prompt[1], pad=pad, bs=bs, back=back, shape=shape)
    return dict(c, name=name) if name else c


def rotary(name=None, N=1, cuts=(32, 16, 16), mixed=False, span=1024, pad=0, H_q=64, H_kv=8, D=128, bs=16,
           interleaved=False, src="bf16", kv="bf16"):
    c = dict(op="rotary", N=N, cut0=cuts[0], cut1=cuts[1], cut2=cuts[2], mixed=mixed, span=span, pad=pad, H_q=H_q,
             H_kv=H_kv, D=D, bs=bs, interleaved=interleaved, src=src, kv=kv)
    return dict(c, name=name) if name else c


def store(name=None, N=1, pool=16, H_kv=8, D=128, bs=16, src="bf16", scaled=False, pad=0):
    c = dict(op="store", N=N, pool=max(pool, N), H_kv=H_kv, D=D, bs=bs, src=src, scaled=scaled, pad=pad)
    return dict(c, name=name) if name else c


def attend(name=None, B=1, q=(1, 1), past=(0, 0), H_q=64, H_kv=8, D=128, bs=16, scaled=True, softcap=0.0, window=0,
           bias=False, prefix=(0, 0), shape=1):
    c = dict(op="attend", B=B, q_min=q[0], q_max=q[1], past_min=past[0], past_max=past[1], H_q=H_q, H_kv=H_kv, D=D,
             bs=bs, scaled=scaled, softcap=float(softcap), window=window, bias=bias, prefix_min=prefix[0],
             prefix_max=prefix[1], shape=shape)
    return dict(c, name=name) if name else c


def _log(rng, lo, hi):
    """A whole number of [lo, hi], spread over its logarithm."""
    return min(hi, max(lo, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def draw(rng):
    op = rng.choice(["tables", "rotary", "store", "attend", "attend"])
    D, bs = rng.choice([64, 128, 128]), rng.choice([16, 32])
    H_kv = rng.choice([1, 2, 3, 4, 8])
    if op == "tables":
        B = _log(rng, 1, 2048)
        if rng.random() < 0.3:
            return tables(B=B, past=(0, _log(rng, 16, 32768 if B <= 64 else 4096)), bs=bs, back=True,
                          shape=rng.randrange(1 << 20))
        return tables(B=B, past=(0, _log(rng, 1, 8191)), new=(0 if B > 15 else 1, rng.choice([1, 1, 4, 16])),
                      prompts=rng.choice([0, 0, rng.randint(0, min(B, 64))]), prompt=(1, _log(rng, 16, 4096)),
                      pad=rng.choice([0, 0, rng.randint(1, 300)]), bs=bs, shape=rng.randrange(1 << 20))
    if op == "rotary":
        half = D // 2
        a = rng.randint(1, half - 2)
        b = rng.randint(1, half - a - 1)
        return rotary(N=_log(rng, 1, 8192), cuts=(a, b, half - a - b), mixed=rng.random() < 0.5,
                      span=_log(rng, 16, 1 << 20), pad=rng.choice([0, 0, 1]), H_q=H_kv * rng.choice([1, 2, 5, 8]),
                      H_kv=H_kv, D=D, bs=bs, interleaved=rng.random() < 0.5, src=rng.choice(["bf16", "f32"]),
                      kv=rng.choice(["bf16", "e4m3"]))
    if op == "store":
        N = _log(rng, 1, 8192)
        return store(N=N, pool=min(8192, N + _log(rng, 1, 4096)), H_kv=H_kv, D=D, bs=bs,
                     src=rng.choice(["bf16", "bf16", "f32"]), scaled=rng.random() < 0.5,
                     pad=rng.choice([0, 0, rng.randint(0, N - 1)]))
    H_q = H_kv * rng.choice([1, 2, 3, 4, 5, 6, 7, 8, 12, 16])
    kind = rng.choice(["decode", "decode", "chunks", "prompts"])
    if kind == "decode":
        B = _log(rng, 1, 128)
        hi = _log(rng, 64, 8191)
        q, past = (1, 1), (hi // 4, hi)
    else:
        B = _log(rng, 1, 16)
        room = 1.0e9 / (B * H_q)                      # padded scores of the plain form, in elements
        hi = _log(rng, 2, max(2, min(2048, int(math.sqrt(room)))))
        q = (max(1, hi // 8), hi)
        past = (0, 0) if kind == "prompts" else (0, _log(rng, 1, max(1, min(8192, int(room / hi) - hi))))
    return attend(B=B, q=q, past=past, H_q=H_q, H_kv=H_kv, D=D, bs=bs, scaled=rng.random() < 0.5,
                  softcap=rng.choice([0.0, 0.0, 30.0, 50.0]), window=rng.choice([0, 0, 0, _log(rng, 16, 2048)]),
                  bias=rng.random() < 0.25, prefix=rng.choice([(0, 0), (0, 0), (1, 300)]),
                  shape=rng.randrange(1 << 20))


def _table_lens(c):
    """(cached, new) tokens of every request, from the case alone."""
    r = random.Random(c["shape"])
    past = [r.randint(c["past_min"], c["past_max"]) for _ in range(c["B"])]
    new = [r.randint(c["new_min"], c["new_max"]) for _ in range(c["B"])]
    for b in r.sample(range(c["B"]), c["prompts"]):
        past[b], new[b] = 0, r.randint(c["prompt_min"], c["prompt_max"])
    return past, new


def _chunk_lens(c):
    """(new tokens, context, prefix) of every sequence, from the case alone."""
    r = random.Random(c["shape"])
    q = [r.randint(c["q_min"], c["q_max"]) for _ in range(c["B"])]
    ctx = [n + r.randint(c["past_min"], c["past_max"]) for n in q]
    return q, ctx, [r.randint(c["prefix_min"], c["prefix_max"]) for _ in range(c["B"])]


# ---------------------------------------------------------------- inputs

def prepare(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(int(seed))
    return {"tables": _prepare_tables, "rotary": _prepare_rotary, "store": _prepare_store,
            "attend": _prepare_attend}[case["op"]](case, gen)


def _randn(gen, *shape):
    return torch.randn(shape, generator=gen, device=DEV)


def _ints(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def _block_tables(gen, lens, bs, width=0, spare=3):
    """Block tables over a shuffled pool (-1 past each sequence), the pool's
    size and its free blocks in a shuffled order."""
    need = torch.tensor([-(-n // bs) for n in lens], device=DEV)
    held, most = int(need.sum()), max(1, width, int(need.max()))
    order = torch.randperm(held + spare, generator=gen, device=DEV)
    first = torch.cumsum(need, 0) - need
    j = torch.arange(most, device=DEV)
    at = (first[:, None] + j).clamp(max=held + spare - 1)
    return torch.where(j < need[:, None], order[at], -1).to(torch.int32), held + spare, order[held:].to(torch.int32)


def _prepare_tables(c, gen):
    past, new = _table_lens(c)
    bs = c["bs"]
    if c["back"]:
        new = [0] * c["B"]
    width = max(-(-(p + n) // bs) for p, n in zip(past, new))
    need = sum(-(-(p + n) // bs) - -(-p // bs) for p, n in zip(past, new))
    spare = need + 17
    table, blocks, free = _block_tables(gen, past, bs, width, spare)
    count = free.numel()
    if c["back"]:                                     # room for every block on the list
        free = torch.cat([free, torch.full((blocks - count,), -1, dtype=torch.int32, device=DEV)])
    r = random.Random(c["shape"] + 1)
    keep = [0 if r.random() < 0.9 else r.randint(0, p) for p in past]   # a few only lose their last tokens
    # the pool that the tables address: its geometry counts here, not what it holds
    pool = torch.empty((blocks, 1, bs, 64), dtype=torch.bfloat16, device=DEV)
    return {"case": c, "table": table, "past": _ints(past), "new": _ints(new), "keep": _ints(keep), "free": free,
            "count": _ints([count]), "pool": pool, "most": sum(new) + c["pad"]}


def _pool(gen, c, blocks):
    """K and V pools; E4M3 codes of values up to about 448 / 64 scales."""
    shape = (blocks, c["H_kv"], c["bs"], c["D"])
    if c["kv"] == "bf16":
        return _randn(gen, *shape).bfloat16(), _randn(gen, *shape).bfloat16()
    return tuple((_randn(gen, *shape) * 64.0).clamp(-448.0, 448.0).to(torch.float8_e4m3fn) for _ in range(2))


def _prepare_rotary(c, gen):
    N, bs, dt = c["N"], c["bs"], torch.bfloat16 if c["src"] == "bf16" else torch.float32
    blocks = -(-N // bs) + 2
    k_cache, v_cache = _pool(gen, c, blocks)
    pos = torch.randint(0, c["span"], (3, N), generator=gen, device=DEV)
    pos[:, : N // 4] = torch.arange(N // 4, device=DEV)            # text: the same along every axis
    slots = torch.randperm(blocks * bs, generator=gen, device=DEV)[:N]
    if c["pad"]:
        slots = torch.where(torch.arange(N, device=DEV) < N - c["pad"], slots, -1)
    cuts, half = (c["cut0"], c["cut1"], c["cut2"]), c["D"] // 2
    axes = [a for a, n in enumerate(cuts) for _ in range(n)]
    if c["mixed"]:                                                 # time, height, width, time, ... while there are some
        left, axes = list(cuts), []
        while len(axes) < half:
            for a in range(3):
                if left[a] > 0:
                    left[a] -= 1
                    axes.append(a)
    f = 10000.0 ** (-torch.arange(0, c["D"], 2, dtype=torch.float64) / c["D"])
    s = {"case": c, "q": _randn(gen, N, c["H_q"], c["D"]).to(dt), "kn": _randn(gen, N, c["H_kv"], c["D"]).to(dt),
         "vn": _randn(gen, N, c["H_kv"], c["D"]).to(dt), "pos": pos, "axes": _ints(axes), "slots": slots,
         "f": f.to(DEV), "k": k_cache, "v": v_cache, "ks": None, "vs": None}
    if c["kv"] == "e4m3":
        s["ks"], s["vs"] = (((0.5 + torch.rand((N, c["H_kv"]), generator=gen, device=DEV)) / 64.0) for _ in range(2))
    return s


def _encoded(x):
    """(codes, scales) of float32 values in groups of 16 along the last axis:
    the scale is the group's largest magnitude / 6 in E4M3 (saturating), a code
    the nearest of 0, 1/2, 1, 3/2, 2, 3, 4, 6 to |value / scale|, ties to the
    even code, with the sign in bit 3.  Codes as int64, scales as float8."""
    g = x.unflatten(-1, (-1, 16))
    s = (g.abs().amax(-1) / 6.0).clamp(max=448.0).to(torch.float8_e4m3fn)
    sv = s.float()[..., None]
    y = torch.where(sv > 0.0, g / sv, 0.0)
    a = y.abs()
    code = ((a > 0.25).long() + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5.0)
            + 8 * torch.signbit(y))
    return code.flatten(-2), s


def _packed(code):
    """Two codes to a byte, the even element in the low half."""
    return (code[..., 0::2] + 16 * code[..., 1::2]).to(torch.uint8)


def _e2m1_pool(gen, blocks, H, bs, D):
    """A pool of quantised normal values with some larger channels."""
    pool = torch.empty((blocks, H, bs, D // 2 + D // 16), dtype=torch.uint8, device=DEV)
    loud = 1.0 + 7.0 * (torch.rand((H, 1, D), generator=gen, device=DEV) > 0.97)
    flat = pool.view(blocks, H, bs * (D // 2 + D // 16))
    step = max(1, (1 << 27) // (H * bs * D))          # blocks at a time
    for b in range(0, blocks, step):
        x = _randn(gen, min(step, blocks - b), H, bs, D) * loud
        code, s = _encoded(x)
        flat[b:b + step, :, :bs * (D // 2)] = _packed(code).flatten(2)
        flat[b:b + step, :, bs * (D // 2):] = s.view(torch.uint8).flatten(2)
    return pool


def _prepare_store(c, gen):
    N, bs, dt = c["N"], c["bs"], torch.bfloat16 if c["src"] == "bf16" else torch.float32
    blocks = -(-c["pool"] // bs)
    loud = 1.0 + 7.0 * (torch.rand((c["H_kv"], c["D"]), generator=gen, device=DEV) > 0.97)
    slots = torch.randperm(blocks * bs, generator=gen, device=DEV)[:N]
    if c["pad"]:
        slots = torch.where(torch.arange(N, device=DEV) < N - c["pad"], slots, -1)
    s = {"case": c, "kn": (_randn(gen, N, c["H_kv"], c["D"]) * loud).to(dt),
         "vn": _randn(gen, N, c["H_kv"], c["D"]).to(dt), "slots": slots,
         "all": torch.arange(blocks * bs, device=DEV), "k": _e2m1_pool(gen, blocks, c["H_kv"], bs, c["D"]),
         "v": _e2m1_pool(gen, blocks, c["H_kv"], bs, c["D"]), "ks": None, "vs": None}
    if c["scaled"]:                                   # values scaled so that the groups' scales use E4M3's range
        s["ks"], s["vs"] = ((0.5 + torch.rand((c["H_kv"],), generator=gen, device=DEV)) / 64.0 for _ in range(2))
    return s


def _prepare_attend(c, gen):
    q_len, ctx, prefix = _chunk_lens(c)
    table, blocks, _ = _block_tables(gen, ctx, c["bs"])
    starts = [0]
    for n in q_len:
        starts.append(starts[-1] + n)
    s = {"case": c, "k": _e2m1_pool(gen, blocks, c["H_kv"], c["bs"], c["D"]),
         "v": _e2m1_pool(gen, blocks, c["H_kv"], c["bs"], c["D"]), "table": table, "max_q": max(q_len),
         "max_ctx": max(ctx), "q": _randn(gen, starts[-1], c["H_q"], c["D"]).bfloat16(), "starts": _ints(starts),
         "ctx": _ints(ctx), "scale": c["D"] ** -0.5, "slopes": None, "prefix": None, "ks": None, "vs": None}
    if c["bias"]:
        s["slopes"] = torch.exp2(-8.0 * torch.arange(1, c["H_q"] + 1, device=DEV) / c["H_q"]).float()
    if c["prefix_max"]:
        s["prefix"] = _ints(prefix)
    if c["scaled"]:
        s["ks"], s["vs"] = (0.5 + torch.rand((c["B"], c["H_kv"]), generator=gen, device=DEV) for _ in range(2))
    return s


# ---------------------------------------------------------------- one pass

def run(state):
    return {"tables": _run_tables, "rotary": _run_rotary, "store": _run_store,
            "attend": _run_attend}[state["case"]["op"]](state)


def _run_tables(s):
    c = s["case"]
    if own:
        import paged_kv_cache_222_gb300 as pkv
        if c["back"]:
            count = pkv.truncate_tables(s["table"], s["past"], s["keep"], s["free"], s["count"], s["pool"])
            return count, s["free"]
        x = pkv.extend_tables(s["table"], s["past"], s["new"], s["free"], s["count"], s["pool"], s["most"])
        return (x.context_lens, x.q_starts, x.slot_mapping, x.positions, x.block_starts, x.free_count, x.lacking,
                s["table"])
    bs, table, past = c["bs"], s["table"], s["past"].long()
    zero = torch.zeros(1, dtype=torch.long, device=DEV)
    if c["back"]:
        first = (s["keep"].long() + bs - 1) // bs
        ends = torch.cumsum((past + bs - 1) // bs - first, 0)
        starts = torch.cat([zero, ends])
        j = torch.arange(s["free"].numel(), device=DEV)            # no more blocks than the list holds
        b = torch.searchsorted(ends, j, right=True).clamp(max=c["B"] - 1)
        live = j < ends[-1]
        ids = table[b, (first[b] + j - starts[b]).clamp(0, table.shape[1] - 1)]
        at = s["count"].long() + ends[-1] - 1 - j
        s["free"][at[live]] = ids[live]
        return s["count"] + ends[-1].to(torch.int32), s["free"]
    new = s["new"].long()
    ctx = past + new
    have = (past + bs - 1) // bs
    ends, block_ends = torch.cumsum(new, 0), torch.cumsum((ctx + bs - 1) // bs - have, 0)
    starts, block_starts = torch.cat([zero, ends]), torch.cat([zero, block_ends])
    t = torch.arange(s["most"], device=DEV)
    b = torch.searchsorted(ends, t, right=True).clamp(max=c["B"] - 1)
    live = t < ends[-1]
    pos = past[b] + t - starts[b]
    blk = pos // bs
    taken = s["count"].long() - 1 - (block_starts[b] + blk - have[b])
    ids = torch.where(blk >= have[b], s["free"][taken.clamp(0, s["free"].numel() - 1)],
                      table[b, blk.clamp(0, table.shape[1] - 1)]).long()
    opened = live & (blk >= have[b]) & (pos % bs == 0)
    table[b[opened], blk[opened]] = ids[opened].to(torch.int32)
    return (ctx.to(torch.int32), starts.to(torch.int32), torch.where(live, ids * bs + pos % bs, -1),
            torch.where(live, pos, -1), block_starts.to(torch.int32), s["count"] - block_ends[-1].to(torch.int32),
            torch.zeros_like(s["count"]), table)


def _turned(x, cos, sin, interleaved):
    half = x.shape[-1] // 2
    if interleaved:
        u, w = x[..., 0::2], x[..., 1::2]
        return torch.stack((u * cos - w * sin, w * cos + u * sin), -1).flatten(-2)
    u, w = x[..., :half], x[..., half:]
    return torch.cat((u * cos - w * sin, w * cos + u * sin), -1)


def _run_rotary(s):
    c = s["case"]
    if own:
        import paged_kv_cache_222_gb300 as pkv
        q = pkv.rotary_append(s["q"], s["kn"], s["vn"], s["pos"], s["f"], s["slots"], s["k"], s["v"], k_scale=s["ks"],
                              v_scale=s["vs"], interleaved=c["interleaved"], axes=s["axes"])
        return q, s["k"], s["v"]
    angle = s["pos"].double()[s["axes"].long()].T * s["f"]
    cos, sin = torch.cos(angle).float()[:, None], torch.sin(angle).float()[:, None]
    q = _turned(s["q"].float(), cos, sin, c["interleaved"]).bfloat16()
    k, v = _turned(s["kn"].float(), cos, sin, c["interleaved"]), s["vn"].float()
    if s["ks"] is not None:
        k = (k / s["ks"][:, :, None]).clamp(-448.0, 448.0)
        v = (v / s["vs"][:, :, None]).clamp(-448.0, 448.0)
    live = s["slots"] >= 0
    slot = s["slots"][live]
    blk, off = slot // c["bs"], slot % c["bs"]
    dt, raw = s["k"].dtype, torch.uint8 if s["k"].dtype == torch.float8_e4m3fn else s["k"].dtype
    s["k"].view(raw)[blk, :, off] = k[live].to(dt).view(raw)
    s["v"].view(raw)[blk, :, off] = v[live].to(dt).view(raw)
    return q, s["k"], s["v"]


def _parts(cache):
    """The code bytes [blocks, H, bs, D / 2] and the scales [blocks, H, bs, D / 16] of an E2M1 pool, as views."""
    nb, H, bs, row = cache.shape
    D = row * 16 // 9
    flat = cache.view(nb, H, bs * row)
    return (flat[:, :, :bs * (D // 2)].view(nb, H, bs, D // 2),
            flat[:, :, bs * (D // 2):].view(nb, H, bs, D // 16))


def _values(codes, scales):
    """Float32 values of code bytes [..., D / 2] and scale bytes [..., D / 16]."""
    code = torch.stack((codes & 15, codes >> 4), -1).flatten(-2)
    m = (code & 7).float()                            # 0, 1/2, then (1 or 3/2) * 2^(0, 1, 2)
    x = torch.where(m < 2.0, 0.5 * m, (1.0 + 0.5 * (code & 1)) * torch.exp2(torch.floor(0.5 * m) - 1.0))
    x = x * (1.0 - 2.0 * (code >> 3))
    s = scales.contiguous().view(torch.float8_e4m3fn).float()
    return (x.unflatten(-1, (-1, 16)) * s[..., None]).flatten(-2)


def _stored(cache, rows, scale, slots):
    """Rows [N, H, D] quantised into their slots."""
    bs = cache.shape[2]
    x = rows.float()
    if scale is not None:
        x = x / scale[:, None]
    code, sc = _encoded(x)
    live = slots >= 0
    blk, off = slots[live] // bs, slots[live] % bs
    codes, scales = _parts(cache)
    codes[blk, :, off] = _packed(code)[live]
    scales[blk, :, off] = sc.view(torch.uint8)[live]


def _read(cache, scale):
    """Every token row of the pool, bfloat16 [tokens, H, D]."""
    x = _values(*_parts(cache))
    if scale is not None:
        x = x * scale[:, None, None]
    return x.permute(0, 2, 1, 3).flatten(0, 1).bfloat16()


def _run_store(s):
    if own:
        import paged_kv_cache_222_gb300 as pkv
        pkv.append(s["kn"], s["vn"], s["slots"], s["k"], s["v"], s["ks"], s["vs"])
        return pkv.read_tokens(s["all"], s["k"], s["v"], s["ks"], s["vs"])
    _stored(s["k"], s["kn"], s["ks"], s["slots"])
    _stored(s["v"], s["vn"], s["vs"], s["slots"])
    return _read(s["k"], s["ks"]), _read(s["v"], s["vs"])


def _rows_of(table, cache):
    """Every token row a table addresses, float32 [B, H, MB * bs, D]."""
    ids = table.long().clamp(min=0)
    codes, scales = _parts(cache)
    x = _values(codes[ids], scales[ids])
    return x.permute(0, 2, 1, 3, 4).flatten(2, 3)


def _run_attend(s):
    c = s["case"]
    if own:
        import paged_kv_cache_222_gb300 as pkv
        return pkv.chunk_attention(s["q"], s["k"], s["v"], s["table"], s["ctx"], s["starts"], s["scale"],
                                   max_q_len=s["max_q"], max_context_len=s["max_ctx"], k_scale=s["ks"],
                                   v_scale=s["vs"], softcap=c["softcap"], window=c["window"], slopes=s["slopes"],
                                   prefix_lens=s["prefix"])
    B, H_q, H, D = c["B"], c["H_q"], c["H_kv"], c["D"]
    G, L = H_q // H, s["max_q"]
    starts, ctx = s["starts"].long(), s["ctx"].long()
    n = starts[1:] - starts[:-1]
    K, V = _rows_of(s["table"], s["k"]), _rows_of(s["table"], s["v"])
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


# ---------------------------------------------------------------- what a pass cannot do without

def work(case):
    return {"tables": _work_tables, "rotary": _work_rotary, "store": _work_store,
            "attend": _work_attend}[case["op"]](case)


def _work_tables(c):
    """Both lengths of every request; a free block's id read and its entry
    written (or the other way round); with new tokens the three per-request
    numbers, the last block's entry and two 64-bit numbers per place of the step."""
    past, new = _table_lens(c)
    bs = c["bs"]
    if c["back"]:
        r = random.Random(c["shape"] + 1)
        keep = [0 if r.random() < 0.9 else r.randint(0, p) for p in past]
        gone = sum(-(-p // bs) - -(-k // bs) for p, k in zip(past, keep))
        return {"bytes": 8 * c["B"] + 8 * gone + 8, "flops": 0}
    need = sum(-(-(p + n) // bs) - -(-p // bs) for p, n in zip(past, new))
    into = sum(1 for p, n in zip(past, new) if p % bs and n)       # requests whose last block has room
    return {"bytes": (8 + 12) * c["B"] + 8 * need + 4 * into + 16 * (sum(new) + c["pad"]) + 20, "flops": 0}


def _work_rotary(c):
    src, dst = (2 if c["src"] == "bf16" else 4), (2 if c["kv"] == "bf16" else 1)
    live = c["N"] - c["pad"]
    return {"bytes": c["N"] * (c["H_q"] * c["D"] * (src + 2) + 24 + 8) + 2 * live * c["H_kv"] * c["D"] * (src + dst),
            "flops": 3 * (c["N"] * c["H_q"] + live * c["H_kv"]) * c["D"]}


def _work_store(c):
    """Live rows read and their codes and scales written; the pool's codes and
    scales read and its values written; a product or quotient per value."""
    src = 2 if c["src"] == "bf16" else 4
    live, pool = c["N"] - c["pad"], -(-c["pool"] // c["bs"]) * c["bs"]
    row = c["H_kv"] * c["D"]
    return {"bytes": 2 * row * (live * (src + 9 / 16) + pool * (9 / 16 + 2)) + 8 * (c["N"] + pool),
            "flops": 2 * row * (live + pool)}


def _work_attend(c):
    """Every query read and output written once, every key and value that some
    query sees read once; two products per query head and visible pair."""
    pairs = seen = rows = 0
    for n, ctx, prefix in zip(*_chunk_lens(c)):
        pos = np.arange(ctx - n, ctx, dtype=np.int64)
        lo = np.maximum(0, pos - c["window"] + 1) if c["window"] else np.zeros_like(pos)
        p = min(prefix, ctx)
        both = np.maximum(0, np.minimum(pos + 1, p) - lo)                 # in the window and in the prefix
        pairs += int((pos + 1 - lo + p - both).sum())
        seen += min(ctx, p + max(0, ctx - max(p, int(lo[0]))))
        rows += n
    return {"bytes": 4 * rows * c["H_q"] * c["D"] + 2 * seen * c["H_kv"] * c["D"] * 9 / 16,
            "flops": 4 * pairs * c["H_q"] * c["D"]}


# ---------------------------------------------------------------- the definition in 64 bits

def exact(case, seed):
    if case["op"] == "tables":
        return None                                   # whole numbers: the plain form has them exactly
    s = prepare(case, seed)
    return {"rotary": _exact_rotary, "store": _exact_store, "attend": _exact_attend}[case["op"]](s)


def _exact_rotary(s):
    """Each pair as a complex number, times e^(i angle) of its axis."""
    c = s["case"]
    half = c["D"] // 2
    angle = torch.stack([s["pos"][a].double() * s["f"][i] for i, a in enumerate(s["axes"].tolist())], 1)
    turn = torch.polar(torch.ones_like(angle), angle)[:, None]
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


_SIZES = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def _exact_pool(cache):
    """Float64 values [tokens, H, D] of an E2M1 pool, byte by byte from a table of all 256."""
    nb, H, bs, row = cache.shape
    D = row * 16 // 9
    flat = cache.reshape(nb, H, -1).long()
    pair = torch.tensor([[(1 - 2 * (h >> 3)) * _SIZES[h & 7] for h in (b & 15, b >> 4)] for b in range(256)],
                        dtype=torch.float64, device=DEV)
    e4m3 = torch.tensor([(-1 if b >> 7 else 1) * (math.nan if b & 127 == 127 else (b & 7) * 2.0 ** -9 if b & 120 == 0
                                                  else (8 + (b & 7)) * 2.0 ** ((b >> 3 & 15) - 10))
                         for b in range(256)], dtype=torch.float64, device=DEV)
    x = pair[flat[:, :, :bs * D // 2]].reshape(nb, H, bs, D // 16, 16)
    x = x * e4m3[flat[:, :, bs * D // 2:]].reshape(nb, H, bs, D // 16, 1)
    return x.reshape(nb, H, bs, D).permute(0, 2, 1, 3).reshape(nb * bs, H, D)


def _exact_quantised(x):
    """Float64 values of rows [N, H, D] after quantisation, by the nearest code: distances in 64 bits."""
    y = x.reshape(x.shape[0], x.shape[1], -1, 16)
    codes = [(8 + m) * 2.0 ** (e - 10) for e in range(1, 16) for m in range(8) if (e, m) != (15, 7)]
    codes = torch.tensor([m * 2.0 ** -9 for m in range(8)] + codes, dtype=torch.float64, device=DEV)
    # the scale: a binary32 quotient, then the nearest E4M3 number, ties to the even code
    want = (y.abs().amax(-1, keepdim=True) / 6.0).float().double().clamp(max=448.0)
    up = torch.searchsorted(codes, want).clamp(1, codes.numel() - 1)
    far, near = codes[up] - want, want - codes[up - 1]
    s = torch.where((far < near) | ((far == near) & (up % 2 == 0)), codes[up], codes[up - 1])
    z = torch.where(s > 0.0, y / s, 0.0).float().double()
    sizes = torch.tensor(_SIZES, dtype=torch.float64, device=DEV)
    up = torch.searchsorted(sizes, z.abs().clamp(max=6.0)).clamp(1, 7)
    far, near = sizes[up] - z.abs().clamp(max=6.0), z.abs().clamp(max=6.0) - sizes[up - 1]
    size = torch.where((far < near) | ((far == near) & (up % 2 == 0)), sizes[up], sizes[up - 1])
    return (torch.copysign(size, z) * s).reshape(x.shape)


def _exact_store(s):
    out = []
    for cache, rows, scale in ((s["k"], s["kn"], s["ks"]), (s["v"], s["vn"], s["vs"])):
        x = rows.double()
        if scale is not None:
            x = (x / scale.double()[:, None]).float().double()
        pool = _exact_pool(cache)
        live = s["slots"] >= 0
        pool[s["slots"][live]] = _exact_quantised(x)[live]
        out.append(pool if scale is None else pool * scale.double()[:, None])
    return tuple(out)


def _exact_attend(s):
    """Sequence by sequence, head by head: softmax over the visible keys."""
    c = s["case"]
    G, bs = c["H_q"] // c["H_kv"], c["bs"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEV)
    starts, ctxs = s["starts"].tolist(), s["ctx"].tolist()
    prefix = s["prefix"].tolist() if s["prefix"] is not None else [0] * c["B"]
    for b, ctx in enumerate(ctxs):
        n = starts[b + 1] - starts[b]
        ids = s["table"][b, :-(-ctx // bs)].long()
        key = torch.arange(ctx, device=DEV)
        pos = torch.arange(ctx - n, ctx, device=DEV)
        d = pos[:, None] - key[None, :]                                    # how far back a key lies
        hidden = (d < 0) if not c["window"] else (d < 0) | (d >= c["window"])
        hidden &= (key >= prefix[b])[None, :]
        for h in range(c["H_kv"]):
            K, V = (_exact_pool(x[ids, h:h + 1])[:ctx, 0] for x in (s["k"], s["v"]))
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
