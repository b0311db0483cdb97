"""Strides of keys, values and queries: what the strides of dimensions of one
say does not matter; the others are honoured or refused."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from speculative_decoding_draft_06_gb300 import dartree as dtl
from tests import cache_ref as ref
from tests.test_gpu_cache import cu, host

pytestmark = pytest.mark.gpu

ONES = [  # R, n, Hkv, strides of K, strides of V
    (1, 5, 2, (1001, 256, 128, 1), (1001, 256, 128, 1)),     # an odd stride between requests, of which there is one
    (1, 5, 2, (2048, 256, 128, 1), (512, 256, 128, 1)),      # different ones
    (3, 1, 2, (512, 301, 128, 1), (512, 8, 128, 1)),         # tokens
    (1, 1, 2, (7, 3, 128, 1), (1, 1, 128, 1)),
    (2, 3, 1, (1024, 136, 5, 1), (1024, 136, 999, 1)),       # heads
    (1, 1, 1, (3, 5, 7, 1), (9, 11, 13, 1)),
]


@pytest.mark.parametrize("case", range(len(ONES)))
def test_strides_of_dimensions_of_one(case):
    R, n, Hkv, ks, vs = ONES[case]
    cache = dtl.KVCache(1, 4, page_tokens=16, Hkv=Hkv, dh=128)
    x, y = (torch.randn(8000, device="cuda").to(torch.bfloat16) for _ in range(2))
    K, V = x.as_strided((R, n, Hkv, 128), ks), y.as_strided((R, n, Hkv, 128), vs)
    table, lens = cu(np.arange(R)[:, None]), cu([0] * R)
    cache.append(0, K, V, table, lens)
    got = cache.read(0, table, lens, n)
    cache.check()
    for a, b in zip(got, (K, V)):
        assert np.array_equal(host(a.double()), ref.values(*ref.quantise(host(b.double()))))


@pytest.mark.parametrize("ks,vs,error", [
    ((1024, 256, 128, 1), (1280, 256, 128, 1), ValueError), ((1024, 256, 128, 1), (1024, 264, 128, 1), ValueError),
    ((1024, 256, 64, 1), (1024, 256, 64, 1), ValueError), ((1024, 512, 256, 2), (1024, 512, 256, 2), ValueError),
    ((1028, 256, 128, 1), (1028, 256, 128, 1), dtl.DartreeError), ((1024, 260, 128, 1), (1024, 260, 128, 1), dtl.DartreeError),
    ((1024, 128, 128, 1), (1024, 128, 128, 1), dtl.DartreeError)])
def test_other_strides_are_refused(ks, vs, error):
    cache = dtl.KVCache(1, 4, page_tokens=16, Hkv=2, dh=128)
    x = torch.zeros(8000, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(error):
        cache.append(0, x.as_strided((2, 3, 2, 128), ks), x.as_strided((2, 3, 2, 128), vs), cu([[0], [1]]), cu([0, 0]))
    cache.check()


def test_queries_strides_of_dimensions_of_one():
    cache = dtl.KVCache(1, 4, page_tokens=16, Hkv=1, dh=128)
    K = torch.randn(1, 9, 1, 128, device="cuda").to(torch.bfloat16)
    table, lens = cu([[0]]), cu([0])
    cache.append(0, K, -K, table, lens)
    lens[0] = 9
    x = torch.randn(4000, device="cuda").to(torch.bfloat16)
    for Hq, st in ((4, (7, 9, 128, 1)), (1, (7, 9, 11, 1)), (4, (2048, 1, 128, 1))):
        Q = x.as_strided((1, 1, Hq, 128), st)
        assert torch.equal(cache.attention(0, Q, table, lens, max_len=9),
                           cache.attention(0, Q.contiguous().clone(), table, lens, max_len=9))
    cache.check()
