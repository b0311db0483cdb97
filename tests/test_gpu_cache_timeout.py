"""A pipeline wait of the attention over the cache that runs out: reported,
nothing hangs or faults, and the next call is right.  Provoked by a limit of
one cycle (a test knob); waits for copies and MMAs in flight keep the full one."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from speculative_decoding_draft_06_gb300 import dartree as dtl
from tests.test_gpu_cache import cu, host
from tests.test_gpu_cache_attention import check_rows, tree_call

pytestmark = pytest.mark.gpu

TIMEOUT = 5


@pytest.mark.parametrize("B,Hq,Hkv,dh,P,lens", [
    (64, 8, 2, 128, 64, [2500]),                 # two row tiles, splits, leftover rows
    (20, 8, 2, 64, 16, [1500, 900]),             # one row tile
    (60, 32, 4, 128, 32, [700, -1, 1300])])      # several CTAs of rows
def test_trees(monkeypatch, B, Hq, Hkv, dh, P, lens):
    g = np.random.default_rng(B)
    lens, n = np.array(lens), np.full(len(lens), B)
    cache, table, vals, masks, m, q = tree_call(g, lens, n, B, Hq, Hkv, dh, P)
    call = lambda: cache.attention(0, q, cu(table), cu(lens), mask=m, n_nodes=cu(n), max_len=2600)  # noqa: E731
    monkeypatch.setenv("DARTREE_WAIT_LIMIT_CYCLES", "1")
    call()
    monkeypatch.delenv("DARTREE_WAIT_LIMIT_CYCLES")
    with pytest.raises(dtl.DartreeError) as e:
        cache.check()
    assert e.value.status == TIMEOUT
    out = call()
    cache.check()
    check_rows(host(out.double()), host(q.double()), lens, n, masks, vals, dh ** -0.5)


@pytest.mark.parametrize("R,Hq,Hkv,P,L", [(64, 16, 8, 64, 9000), (2, 8, 8, 64, 40000), (1, 8, 8, 128, 8000)])
def test_single_tokens(monkeypatch, R, Hq, Hkv, P, L):
    """One split, a cluster's, the workspace's: keys that memory has to bring."""
    dh, per = 128, -(-L // P)
    cache = dtl.KVCache(1, R * per, page_tokens=P, Hkv=Hkv, dh=dh)
    cache.pool.random_(0, 0x60)
    table = cu(np.random.default_rng(0).permutation(R * per).reshape(R, per))
    q = torch.randn(R, 1, Hq, dh, device="cuda").to(torch.bfloat16)
    lens = cu(np.full(R, L))
    call = lambda: cache.attention(0, q, table, lens, max_len=L)  # noqa: E731
    want = call()
    cache.check()
    monkeypatch.setenv("DARTREE_WAIT_LIMIT_CYCLES", "1")
    torch.empty(200 << 20, dtype=torch.uint8, device="cuda").fill_(1)   # (what is in L2 arrives too soon)
    call()
    monkeypatch.delenv("DARTREE_WAIT_LIMIT_CYCLES")
    with pytest.raises(dtl.DartreeError) as e:
        cache.check()
    assert e.value.status == TIMEOUT
    assert torch.equal(call(), want)
    cache.check()
