"""Sizes beyond the C ABI's 32 bits are refused by the compiled entry with an
ordinary exception, with the interpreter's lock held; later calls and other
threads go on."""

import threading

import pytest
import torch

import paged_kv_cache_222_gb300 as pkv

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda", 0)
TOO_MANY = 2 ** 31


def _caches():
    kc = torch.zeros((4, 2, 16, 128), dtype=torch.bfloat16, device=DEV)
    return kc, torch.zeros_like(kc)


def _ids(*shape):
    return torch.zeros(shape, dtype=torch.int32, device=DEV)


def _rotary_with_too_many_heads():
    kc, vc = _caches()
    q = torch.empty((0, TOO_MANY, 128), dtype=torch.bfloat16, device=DEV)  # no elements
    k = torch.empty((0, 2, 128), dtype=torch.bfloat16, device=DEV)
    none = torch.empty(0, dtype=torch.int64, device=DEV)
    pkv.rotary_append(q, k, k, none, pkv.rotary_frequencies(128, device=DEV), none, kc, vc)


def _chunk_with_too_many_heads():
    kc, vc = _caches()
    q = torch.empty((0, TOO_MANY, 128), dtype=torch.bfloat16, device=DEV)
    pkv.chunk_attention(q, kc, vc, _ids(1, 2), _ids(1), _ids(2), 0.1)


def _chunk_with_too_wide_a_table():
    kc, vc = _caches()
    q = torch.empty((0, 4, 128), dtype=torch.bfloat16, device=DEV)
    pkv.chunk_attention(q, kc, vc, _ids(0, TOO_MANY), _ids(0), _ids(1), 0.1)


def _compact_with_too_wide_a_table():
    kc, vc = _caches()
    pkv.compact_tokens(kc, vc, _ids(0, TOO_MANY), _ids(0), _ids(1))


@pytest.mark.parametrize("call", [_rotary_with_too_many_heads, _chunk_with_too_many_heads,
                                  _chunk_with_too_wide_a_table, _compact_with_too_wide_a_table])
def test_too_large_sizes_are_refused(call):
    ticks = []
    stop = threading.Event()

    def tick():  # runs Python code all the while
        while not stop.is_set():
            ticks.append(1)
            stop.wait(0.001)

    t = threading.Thread(target=tick)
    t.start()
    try:
        for _ in range(3):
            with pytest.raises(ValueError):
                call()
    finally:
        stop.set()
        t.join(10)
    assert not t.is_alive() and ticks
    # the thread still owns its state: an ordinary call works
    kc, vc = _caches()
    k = torch.ones((1, 2, 128), dtype=torch.bfloat16, device=DEV)
    zero = torch.zeros(1, dtype=torch.int64, device=DEV)
    out = pkv.rotary_append(k, k, k, zero, pkv.rotary_frequencies(128, device=DEV), zero, kc, vc)
    assert torch.equal(out, k) and torch.all(kc[0, :, 0] == 1)
    assert pkv.device_error(DEV) == 0
