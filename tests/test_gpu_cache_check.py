"""KVCache.check: what calls on any stream have flagged."""
from __future__ import annotations

import pytest
import torch

from speculative_decoding_draft_06_gb300 import dartree as dtl
from tests.test_gpu_cache import cu

pytestmark = pytest.mark.gpu


def test_check_waits_for_other_streams():
    """A bad call that another stream has not come to yet is not missed."""
    cache = dtl.KVCache(1, 4, page_tokens=64, Hkv=2, dh=128)
    K = torch.zeros(1, 2, 2, 128, dtype=torch.bfloat16, device="cuda")
    table, lens = cu([[-1]]), cu([0])
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(100_000_000)                   # some 50 ms
    cache.append(0, K, K, table, lens, stream=side)
    with pytest.raises(dtl.DartreeError):
        cache.check()
    cache.check()
