"""E2M1 caches whose byte offsets pass 2^32: what happens in the last blocks is
what happens in the first ones of a small cache, bit for bit."""

import pytest
import torch

import paged_kv_cache_222_gb300 as pkv

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda", 0)


@pytest.mark.parametrize("src", [torch.bfloat16, torch.float32])
def test_far_blocks(src):
    nb, near, bs, H, D, n = 520_000, 12, 16, 8, 128, 150
    assert nb * H * bs * 72 > 1 << 32
    far = nb - near
    g = torch.Generator(device=DEV).manual_seed(3)
    big = [pkv.e2m1_cache(nb, H, bs, D, device=DEV) for _ in range(2)]
    small = [pkv.e2m1_cache(near, H, bs, D, device=DEV) for _ in range(2)]
    for c in big + small:
        c[-near:] = 0
    big[0][:near], big[1][:near] = 7, 7               # where offsets cut to 32 bits would lead
    q, k, v = (torch.randn((n, h, D), generator=g, device=DEV).to(src) for h in (16, H, H))
    slots = torch.randperm(near * bs, generator=g, device=DEV)[:n]
    pos = torch.arange(n, device=DEV)
    f = pkv.rotary_frequencies(D, device=DEV)

    def both(run):
        run(small[0], small[1], slots, 0)
        run(big[0], big[1], slots + far * bs, far)
        assert pkv.device_error(DEV) == 0
        assert all(torch.equal(b[far:], s) for b, s in zip(big, small))

    both(lambda kc, vc, s, first: pkv.append(k, v, s, kc, vc))
    got = [pkv.read_tokens(s, *c) for s, c in ((slots, small), (slots + far * bs, big))]
    assert all(torch.equal(a, b) and a.any() for a, b in zip(*got))
    both(lambda kc, vc, s, first: pkv.rotary_append(q, k, v, pos, f, s, kc, vc))
    keep = torch.arange(0, near * bs, 3, dtype=torch.int32, device=DEV)
    starts = torch.tensor([0, keep.numel()], dtype=torch.int32, device=DEV)
    table = torch.randperm(near, generator=g, device=DEV).to(torch.int32)[None]
    both(lambda kc, vc, s, first: pkv.compact_tokens(kc, vc, table + first, keep, starts))
    ids = torch.tensor([[3], [5]], dtype=torch.int32, device=DEV)
    both(lambda kc, vc, s, first: pkv.copy_blocks(kc, vc, ids[0] + first, ids[1] + first))
    assert (big[0][:near] == 7).all() and (big[1][:near] == 7).all()


@pytest.mark.parametrize("n,H,D,bs", [(5000, 8, 128, 16), (40_001, 3, 64, 32)])
@pytest.mark.parametrize("src", [torch.bfloat16, torch.float32])
def test_more_rows_than_a_grid(src, n, H, D, bs):
    # CTAs that take rows in turn write and read what calls of a few rows do
    g = torch.Generator(device=DEV).manual_seed(4)
    nb = -(-n // bs) + 3
    k, v = (torch.randn((n, H, D), generator=g, device=DEV).to(src) for _ in range(2))
    slots = torch.randperm(nb * bs, generator=g, device=DEV)[:n]
    slots[::97] = -1
    one, few = ([pkv.e2m1_cache(nb, H, bs, D, device=DEV).zero_() for _ in range(2)] for _ in range(2))
    pkv.append(k, v, slots, *one)
    for i in range(0, n, 1000):
        pkv.append(k[i:i + 1000].contiguous(), v[i:i + 1000].contiguous(), slots[i:i + 1000].contiguous(), *few)
    assert all(torch.equal(a, b) and a.any() for a, b in zip(one, few))
    got = pkv.read_tokens(slots, *one, dtype=src)
    want = [pkv.read_tokens(slots[i:i + 1000].contiguous(), *one, dtype=src) for i in range(0, n, 1000)]
    assert all(torch.equal(a, torch.cat(b)) and a.any() for a, b in zip(got, zip(*want)))
    assert pkv.device_error(DEV) == 0
