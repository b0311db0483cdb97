"""dartree_cache_copy_pages with thousands of pairs, some of them refused."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from speculative_decoding_draft_06_gb300 import dartree as dtl
from tests.test_gpu_cache import BAD, cu, host

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("n", [300, 5000, 9001])
def test_many_pairs(n):
    g = np.random.default_rng(n)
    pages, layers = 3 * n, 2
    cache = dtl.KVCache(layers, pages, page_tokens=16, Hkv=1, dh=64)
    cache.pool.random_(0, 256)
    pool = host(cache.pool)
    order = g.permutation(pages)
    src, dst = g.choice(order[:n], n), order[n:2 * n].copy()
    for k, bad in enumerate((0, n // 3, n - 1)):           # a destination of a later pair, of an earlier one; a source
        dst[bad] = dst[(bad + 7 * k + 1) % n] if k < 2 else src[5]
    src[n // 2], dst[n // 5] = -1, pages
    want, flagged, seen = pool.copy(), False, set()
    sources = set(src.tolist())
    for s, d in zip(src.tolist(), dst.tolist()):
        ok = 0 <= s < pages and 0 <= d < pages and d not in sources and d not in seen
        seen.add(d)
        flagged |= not ok
        if ok:
            want[:, d] = pool[:, s]
    cache.copy_pages(cu(src), cu(dst))
    assert np.array_equal(host(cache.pool), want)
    assert flagged and int(cache.err.item()) == BAD
