"""Nodes of a tree that nothing has written and no row sees -- a call without
sizes on trees smaller than B -- in a pool whose bytes are e4m3's NaN."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from speculative_decoding_draft_06_gb300 import dartree as dtl
from speculative_decoding_draft_06_gb300 import inputs as I
from tests import cache_ref as ref
from tests.test_gpu_cache import cu, host, tables
from tests.test_gpu_cache_attention import check_rows
from tests.test_gpu_verify import ancestor_mask

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("byte", [0x7F, 0xFF])
@pytest.mark.parametrize("B,n,Hq,Hkv,dh,P,L", [
    (3, 1, 4, 2, 128, 64, 61), (7, 4, 2, 1, 64, 16, 130), (15, 2, 8, 8, 128, 32, 700), (3, 2, 16, 4, 64, 128, 0),
    (40, 17, 8, 2, 128, 64, 200), (64, 30, 8, 2, 128, 16, 1000), (90, 64, 4, 2, 64, 64, 5), (128, 100, 16, 4, 128, 64, 3000)])
def test_nodes_that_nothing_has_written(byte, B, n, Hq, Hkv, dh, P, L):
    g = np.random.default_rng(B + byte)
    R = 2
    lens = np.array([L, L // 3])
    table, refs = tables(g, -(-(lens + B) // P), 2 * (-(-(L + B) // P)) + 2, -(-(L + B) // P))
    cache = dtl.KVCache(1, len(refs), page_tokens=P, Hkv=Hkv, dh=dh, refs=cu(refs))
    cache.pool.fill_(byte)
    masks = np.stack([ancestor_mask(I.random_tree(g, B, n)["parent"], n, B) for _ in range(R)])
    vals = []
    for r in range(R):
        x = [torch.from_numpy(g.standard_normal((1, lens[r] + n, Hkv, dh))).to(torch.bfloat16) for _ in range(2)]
        cache.append(0, x[0].cuda(), x[1].cuda(), cu(table[r:r + 1]), cu([0]))
        # what is not written is not seen: zeros stand for it here
        vals.append(tuple(np.concatenate([ref.values(*ref.quantise(y[0].double().numpy())), np.zeros((B - n, Hkv, dh))])
                          for y in x))
    q = torch.from_numpy(g.standard_normal((R, B + 1, Hq, dh)) * 2).to(torch.bfloat16)
    out = cache.attention(0, q.cuda(), cu(table), cu(lens), mask=torch.from_numpy(masks.view(np.int32)).cuda(), max_len=L + B)
    cache.check()
    check_rows(host(out.double()), q.double().numpy(), lens, [B, B], masks, vals, dh ** -0.5)
