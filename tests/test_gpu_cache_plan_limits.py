"""A page plan whose maps end at the largest number of tokens."""
from __future__ import annotations

import pytest
import torch

from speculative_decoding_draft_06_gb300 import dartree as dtl
from tests.test_gpu_cache import cu, host

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T", [2 ** 31 - 1024, 2 ** 31 - 1023, 2 ** 31 - 1])
def test_the_longest_maps(T):
    """Two tokens, and -1 behind them to the end of maps of up to 2^31 - 1 entries."""
    cache = dtl.KVCache(1, 4, page_tokens=16, Hkv=1, dh=64)
    table, lens = cu([[-1, -1]]), cu([15])
    out = cache.plan(table, lens, cu([2]), max_tokens=T, offset=0)
    cache.check()
    assert host(out["ok"]).tolist() == [1] and host(out["start"]).tolist() == [0, 2]
    assert host(table).tolist() == [[0, 1]] and host(cache.refs).tolist() == [1, 1, 0, 0]
    for name, want in (("row", [0, 0, -1]), ("pos", [15, 16, -1]), ("slot", [15, 16, -1])):
        assert host(out[name][:3]).tolist() == want
        assert int(torch.max(out[name][2:])) == int(torch.min(out[name][2:])) == -1
