"""dartree_cache_commit where lengths and positions end: 2^31 - 1."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from speculative_decoding_draft_06_gb300 import dartree as dtl
from tests.test_gpu_cache import BAD, cu, host

pytestmark = pytest.mark.gpu

TOP = 2 ** 31 - 1


def test_a_length_that_would_wrap_is_left():
    cache = dtl.KVCache(2, 4, page_tokens=16, Hkv=1, dh=64)
    table = cu([[0], [1], [2]])
    lens = cu([TOP, TOP - 1, 5])
    nodes, none = cu([[-1, -1], [-1, -1], [1, 3]]), cu([0, 0, 2])
    cache.commit(table, lens, nodes, none, extra=1)
    assert host(lens).tolist() == [TOP, TOP, 8] and int(cache.err.item()) == BAD
    cache.err.zero_()
    cache.commit(table, lens, nodes, cu([0, 0, 0]), extra=0)
    assert host(lens).tolist() == [TOP, TOP, 8]
    cache.check()
    cache.commit(table, lens, nodes, cu([0, 0, 0]), extra=TOP)
    assert host(lens).tolist() == [TOP, TOP, 8] and int(cache.err.item()) == BAD


def test_positions_past_31_bits_are_refused():
    """A page table wide enough for them."""
    P, width = 128, 2 ** 24 + 1
    cache = dtl.KVCache(1, 2, page_tokens=P, Hkv=1, dh=64)
    cache.pool.copy_(torch.randint(0, 255, cache.pool.shape, dtype=torch.uint8))
    pool = cache.pool.clone()
    table = torch.zeros(1, width, dtype=torch.int32, device="cuda")
    table[0, -2:] = 1
    for node in (20, TOP - 1):
        lens = cu([TOP - 10])
        cache.commit(table, lens, cu([[node]]), cu([1]))
        assert host(lens).tolist() == [TOP - 10] and int(cache.err.item()) == BAD
        assert torch.equal(cache.pool, pool)
        cache.err.zero_()
    lens = cu([TOP - 10])
    cache.commit(table, lens, cu([[4]]), cu([1]))        # positions 2^31 - 11 and - 7: one page's
    cache.check()
    assert host(lens).tolist() == [TOP - 9]
    got = host(cache.pool)[0, 1].reshape(-1)
    half = P * 32
    assert np.array_equal(got[117 * 32:118 * 32], host(pool)[0, 1].reshape(-1)[121 * 32:122 * 32])
    assert np.array_equal(got[half + 117 * 4:half + 118 * 4], host(pool)[0, 1].reshape(-1)[half + 121 * 4:half + 122 * 4])
