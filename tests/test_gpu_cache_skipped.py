"""What a call leaves out -- requests with negative lengths, rows behind a
tree, tokens behind a count -- is zero in an output that the call makes, and
as it was in one that it is given."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from tests.test_gpu_cache import cu, host
from tests.test_gpu_cache_attention import check_rows, filled, tree_call

pytestmark = pytest.mark.gpu


def poisoned(call, *shapes):
    """call() where the allocator's free blocks of these bf16 shapes hold
    NaN."""
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    x = [torch.full(s, float("nan"), dtype=torch.bfloat16, device="cuda") for s in shapes]
    del x
    return call()


@pytest.mark.parametrize("Hq,max_len", [(8, 300), (16, 300), (24, 300), (4, 20000)])
def test_single_tokens_of_skipped_requests(Hq, max_len):
    """One split, splits in a cluster and in the workspace; 24 heads over 1 is
    the tensor-core kernel's."""
    g = np.random.default_rng(Hq)
    Hkv = 1 if Hq == 24 else 2
    lens = np.array([50, -1, 0, 290, -7])
    cache, table, vals = filled(g, lens, 0, 64, Hkv, 128)
    q = torch.from_numpy(g.standard_normal((5, 1, Hq, 128))).to(torch.bfloat16).cuda()
    O = poisoned(lambda: cache.attention(0, q, cu(table), cu(lens), max_len=max_len), q.shape)
    check_rows(host(O.double()), host(q.double()), lens, [0] * 5, None, vals, 128 ** -0.5)
    assert not host(O.float())[[1, 2, 4]].any()
    out = torch.full(q.shape, 5.0, dtype=torch.bfloat16, device="cuda")
    cache.attention(0, q, cu(table), cu(lens), max_len=max_len, out=out)
    assert (host(out.float())[[1, 4]] == 5.0).all() and torch.equal(out[[0, 2, 3]], O[[0, 2, 3]])
    cache.check()


@pytest.mark.parametrize("B,Hq,Hkv,dh", [(5, 4, 2, 128), (40, 8, 2, 64), (70, 8, 2, 128), (150, 4, 2, 64)])
def test_trees_smaller_than_their_rows(B, Hq, Hkv, dh):
    g = np.random.default_rng(B)
    lens, n = np.array([100, 30, -1, 77, 200]), np.array([B, 0, B, min(B, 64 * Hkv // Hq), B // 2])
    cache, table, vals, masks, m, q = tree_call(g, lens, n, B, Hq, Hkv, dh, 32)
    sizes = n.copy()
    sizes[3] = -1                                        # a size below zero: skipped as well
    top = int((np.maximum(lens, 0) + n).max())
    call = lambda **kw: cache.attention(0, q, cu(table), cu(lens), mask=m, n_nodes=cu(sizes), max_len=top, **kw)  # noqa: E731
    O = poisoned(call, q.shape)
    x = host(O.double())
    live = np.array([r for r in range(5) if lens[r] >= 0 and sizes[r] >= 0])
    check_rows(x[live], host(q.double())[live], lens[live], n[live], masks[live], [vals[r] for r in live], dh ** -0.5)
    assert not x[[2, 3]].any()
    out = torch.full(q.shape, 5.0, dtype=torch.bfloat16, device="cuda")
    call(out=out)
    y = host(out.double())
    assert (y[[2, 3]] == 5.0).all()
    for r in live:
        assert not x[r, n[r] + 1:].any() and (y[r, n[r] + 1:] == 5.0).all()
        assert np.array_equal(x[r, :n[r] + 1], y[r, :n[r] + 1])
    cache.check()
    if B == 5:                                           # no sizes (nodes without pages are flagged): skipped requests only
        O = poisoned(lambda: cache.attention(0, q, cu(table), cu(lens), mask=m, max_len=top), q.shape)
        assert not host(O.float())[2].any()


@pytest.mark.parametrize("dh", [64, 128])
def test_read_of_skipped_rows(dh):
    g = np.random.default_rng(dh)
    lens = np.array([40, -1, 3, 20])
    cache, table, vals = filled(g, lens, 13, 16, 3, dh)
    shape = (4, 13, 3, dh)
    for count in (None, np.array([13, 13, 0, 7])):
        c = None if count is None else cu(count)
        got = poisoned(lambda: cache.read(0, cu(table), cu(lens), 13, count=c), shape, shape)
        out = tuple(torch.full(shape, 5.0, dtype=torch.bfloat16, device="cuda") for _ in range(2))
        cache.read(0, cu(table), cu(lens), 13, count=c, out=out)
        for which, (x, y) in enumerate(zip(got, out)):
            for r in range(4):
                k = 0 if lens[r] < 0 else 13 if count is None else count[r]
                if k:
                    assert np.array_equal(host(x[r, :k].double()), vals[r][which][lens[r]:lens[r] + k])
                assert torch.equal(x[r, :k], y[r, :k])
                assert not host(x[r, k:].float()).any() and (host(y[r, k:].float()) == 5.0).all()
    cache.check()
