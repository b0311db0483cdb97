"""Attention over the cache with millions of query heads to a key/value head."""
from __future__ import annotations

import pytest
import torch

from speculative_decoding_draft_06_gb300 import dartree as dtl
from tests.test_gpu_cache import cu

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("g", [255, 256, 4099, 2 ** 22 + 3, 2 ** 23 - 300, 2 ** 23 + 8])
@pytest.mark.parametrize("window, rows", [(None, 1), (5, 1), (5, 2)])
def test_large_groups(g, window, rows):
    """Every head of a row that sees one token has that token's value, exactly; the
    second row of a chain, whose keys are equal, the mean of two values."""
    cache = dtl.KVCache(1, 1, page_tokens=16, Hkv=2, dh=64)
    table, lens = cu([[0]]), cu([1])
    cache.refs.fill_(1)
    x = torch.zeros(1, 2, 2, 64)
    x[0, 0], x[0, 1] = 1.0, 3.0
    x[0, :, 1] *= 2
    x = x.to(torch.bfloat16).cuda()
    cache.append(0, torch.ones_like(x), x, table, cu([0]))
    Q = torch.ones(1, rows, 2 * g, 64, dtype=torch.bfloat16, device="cuda")
    if window is None:
        if 2 * (-(-g // 256)) > 65535:
            with pytest.raises(dtl.DartreeError):
                cache.attention(0, Q, table, lens, max_len=2)
            return
        out = cache.attention(0, Q, table, lens, max_len=2)
    else:
        out = cache.window_attention(0, Q, table, lens, max_len=2, window=window)
    cache.check()
    held = cache.read(0, table, cu([0]), 2)[1][0].float()  # (what 4 bits hold of x)
    for h in range(2):
        mine = out[0, :, h * g:(h + 1) * g]
        assert bool((mine[0] == held[0, h, 0]).all())
        assert bool((mine[1:] == ((held[0, h, 0] + held[1, h, 0]) / 2).to(torch.bfloat16)).all())
