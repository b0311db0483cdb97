"""Attention over the 4-bit cache at the ends of the types' ranges: queries
near the largest and smallest bf16 numbers, scales that move the scores to
where fp32 has few bits left behind the point."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from speculative_decoding_draft_06_gb300 import inputs as I
from tests.test_gpu_cache import cu, host
from tests.test_gpu_cache_attention import check_rows, filled
from tests.test_gpu_verify import ancestor_mask

pytestmark = pytest.mark.gpu


def setup(g, B, dh, ks=1.0):
    lens, n = np.array([200, 77]), np.array([B, max(0, B - 3)])
    masks = np.stack([ancestor_mask(I.random_tree(g, max(B, 1), max(1, int(k)))["parent"], int(k), max(B, 1)) for k in n])
    cache, table, vals = filled(g, lens, n, 64, 2, dh, ks=ks)
    kw = dict(mask=torch.from_numpy(masks.view(np.int32)).cuda(), n_nodes=cu(n)) if B else {}
    return lens, n, masks, cache, cu(table), vals, kw


@pytest.mark.parametrize("B,dh", [(0, 128), (0, 64), (3, 128), (40, 64), (40, 128), (100, 128)])
@pytest.mark.parametrize("e", [100, 117, 126, -100, -113, -117, -126])
def test_queries_at_the_ends_of_their_range(B, dh, e):
    """Rows of about 2^e, with a scale that brings the scores back to ordinary
    ones, and with each row of another size."""
    g = np.random.default_rng(abs(e) + B)
    lens, n, masks, cache, table, vals, kw = setup(g, B, dh)
    x = np.clip(g.standard_normal((2, B + 1, 8, dh)), -3.5, 3.5)
    for spread in (0, 1):
        if spread:
            x = x * 2.0 ** (-np.sign(e) * g.integers(0, 12, (2, B + 1, 8, 1)))
        q = (torch.from_numpy(x).double() * 2.0 ** min(e, 126)).to(torch.bfloat16)
        assert torch.isfinite(q).all()
        scale = 0.25 * 2.0 ** -e
        out = cache.attention(0, q.cuda(), table, cu(lens), max_len=300, scale=scale, **kw)
        cache.check()
        check_rows(host(out.double()), q.double().numpy(), lens, n, masks, vals, scale)


@pytest.mark.parametrize("B", [0, 3, 40])
@pytest.mark.parametrize("ks,e", [(-64, -100), (-64, -60), (64, -126), (64, 40), (0, -126), (-64, 126)])
def test_factors_at_the_ends_of_their_range(B, ks, e):
    """Keys in units of 2^-64 and 2^64 with queries whose scores vanish, or all
    but vanish: what is not seen stays unseen."""
    g = np.random.default_rng(B + abs(ks) + abs(e))
    lens, n, masks, cache, table, vals, kw = setup(g, B, 128, 2.0 ** ks)
    q = (torch.from_numpy(np.clip(g.standard_normal((2, B + 1, 8, 128)), -3, 3)).double() * 2.0 ** min(e, 126)).to(torch.bfloat16)
    scale = 2.0 ** -100 if ks + e > 0 else 128 ** -0.5
    out = cache.attention(0, q.cuda(), table, cu(lens), max_len=300, scale=scale, **kw)
    cache.check()
    check_rows(host(out.double()), q.double().numpy(), lens, n, masks, vals, scale)
