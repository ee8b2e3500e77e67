"""extend_tables: a step that was refused as a whole shows in what it leaves on
the device, whatever the reason, so that a captured step's next kernels can
tell it from one that went through."""

import numpy as np
import pytest
import torch

import paged_kv_cache_222_gb300 as pkv
from oracle import tables as OT

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda", 0)
BS = 16


def up(x, dt=torch.int32):
    return torch.as_tensor(np.asarray(x)).to(dt).to(DEV)


def step(past, new, count, free, most, out=None):
    """The outputs, the table before and after, and the error word."""
    mb = max(1, *(-(-(p + n) // BS) for p, n in zip(past, new)))
    table = np.arange(len(past) * mb, dtype=np.int32).reshape(len(past), mb)
    nb = table.size + len(free) + 5
    t = up(table)
    x = pkv.extend_tables(t, up(past), up(new), up(free), up([count]),
                          torch.empty((nb, 1, BS, 64), dtype=torch.uint8, device=DEV), most, out)
    want = OT.extend(table, past, new, free, count, BS, most, nb)
    for g, w in zip((t, x.context_lens, x.q_starts, x.slot_mapping, x.positions, x.block_starts), want):
        assert np.array_equal(g.cpu().numpy(), w)
    assert (x.free_count.item(), x.lacking.item()) == (want[6], want[7])
    return x, pkv.device_error(DEV)


# held and new tokens with and without a block to be taken; one launch and two
REQUESTS = pytest.mark.parametrize("past,new", [([5], [3]), ([5, 0, 31], [3, 0, 1]), ([10, 20], [20, 6]),
                                                ([15] * 700, [1] * 700), ([16] * 700, [1] * 700), ([0], [4000])],
                                   ids=["no block", "no block of three", "blocks", "700 tokens", "700 blocks", "prompt"])


@REQUESTS
def test_more_tokens_than_places(past, new):
    free = np.arange(10_000, 11_000, dtype=np.int32)
    need = sum(-(-(p + n) // BS) - -(-p // BS) for p, n in zip(past, new))
    for most in (sum(new) - 1, 0):
        x, err = step(past, new, len(free), free, most)
        assert err == 3 and x.lacking.item() == -1
        x, err = step(past, new, 0, free, most)          # too few blocks as well: those are told
        assert err == 3 and x.lacking.item() == (need if need else -1)


@REQUESTS
def test_a_count_that_is_none(past, new):
    free = np.arange(10_000, 10_800, dtype=np.int32)
    need = sum(-(-(p + n) // BS) - -(-p // BS) for p, n in zip(past, new))
    for count in (-1, len(free) + 1, 2 ** 31 - 1, -2 ** 31):
        x, err = step(past, new, count, free, sum(new) + 3)
        assert err == 2 and x.lacking.item() == (need if need else -1) and x.free_count.item() == count


@REQUESTS
def test_a_step_that_goes_through_lacks_nothing(past, new):
    free = np.arange(1000, dtype=np.int32)
    x, err = step(past, new, len(free), free, sum(new))
    assert err == 0 and x.lacking.item() == 0
    x, err = step(past, [0] * len(new), len(free), free, 0)    # nothing asked for
    assert err == 0 and x.lacking.item() == 0


def test_a_request_that_gets_none_beside_others():
    # refused alone: the step goes through, the request's part of it is empty
    free = np.arange(100, dtype=np.int32)
    x, err = step([5, 7, 9], [3, -1, 2], 100, free, 20)
    assert err == 3 and x.lacking.item() == 0 and x.q_starts.tolist() == [0, 3, 3, 5]


def test_seen_from_a_captured_step():
    # a step whose next kernel keeps a number on the device only if it went through
    past, new, count = up([5]), up([3]), up([100])
    free, t = up(np.arange(100)), up([[7, 8, 9]])
    cache = torch.empty((200, 1, BS, 64), dtype=torch.uint8, device=DEV)
    done = torch.zeros(1, dtype=torch.int32, device=DEV)
    x = pkv.extend_tables(t, past, new, free, count, cache, 4)

    def forward():
        pkv.extend_tables(t, past, new, free, count, cache, 4, out=x)
        done.add_((x.lacking == 0).int())

    forward()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        forward()
    for n, goes in ((3, 1), (5, 0), (4, 1), (40, 0), (1, 1)):
        new.fill_(n)
        done.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert done.item() == goes, n
        assert pkv.device_error(DEV) == (0 if goes else 3) and x.context_lens.item() == (5 + n if goes else 5)
