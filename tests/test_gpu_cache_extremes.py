"""Attention over the 4-bit cache at the ends of the types' ranges: queries
near the largest and smallest bf16 numbers, scales that move the scores to
where fp32 has few bits left behind the point."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from speculative_decoding_draft_06_gb300 import inputs as I
from tests import cache_ref as ref
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


@pytest.mark.parametrize("B,dh,Hq,lens", [(0, 128, 8, (200, 77)), (0, 64, 2, (9000, 77)), (5, 128, 8, (200, 77)),
                                          (40, 64, 8, (200, 77)), (70, 128, 8, (3000, 500))])
@pytest.mark.parametrize("scale", [1e5, 1e7, 1e9, 1e12, 1e20, 1e38])
def test_scores_beyond_24_bits(scale, B, dh, Hq, lens):
    """Scores so large that fp32 has no bits left behind the point: the softmax
    is one-hot, or shared by keys whose scores are equal.  Scores here are
    multiples of 2^-12 below 2^12 and so exact, and so is their order."""
    g = np.random.default_rng(B + int(np.log10(scale)))
    lens, Hkv = np.array(lens), 2
    n = np.array([B, max(0, B - 3)])
    masks = np.stack([ancestor_mask(I.random_tree(g, max(B, 1), max(1, int(k)))["parent"], int(k), max(B, 1)) for k in n])
    cache, table, vals = filled(g, lens, n, 64, Hkv, dh)
    # keys of few values each (codes exact: a block's scale is 1), many ties
    for r in range(2):
        K = g.choice([0.0, 0.5, 1.0, -1.0, 2.0], (1, lens[r] + n[r], Hkv, dh)) * (g.random((1, lens[r] + n[r], Hkv, dh)) < 0.1)
        K[..., ::16] = 6.0
        x = torch.from_numpy(K).to(torch.bfloat16)
        V = g.standard_normal(K.shape)
        v = torch.from_numpy(V).to(torch.bfloat16)
        cache.append(0, x.cuda(), v.cuda(), cu(table[r:r + 1]), cu([0]))
        vals[r] = (K[0], ref.values(*ref.quantise(v.double().numpy()))[0])
    q = torch.from_numpy(g.choice([-2.0, -0.25, 0.0, 2.0 ** -11, 1.0, 1.0], (2, B + 1, Hq, dh))).to(torch.bfloat16)
    q[..., 0] = 1.0
    kw = dict(mask=torch.from_numpy(masks.view(np.int32)).cuda(), n_nodes=cu(n)) if B else {}
    out = cache.attention(0, q.cuda(), cu(table), cu(lens), max_len=int((lens + n).max()), scale=scale, **kw)
    cache.check()
    O = host(out.double())
    for r in range(2):
        L, k, (K, V) = int(lens[r]), int(n[r]), vals[r]
        see = np.zeros((k + 1, L + k), bool)
        see[:, :L] = True
        for i in range(k):
            for j in range(k):
                see[i + 1, L + j] = (int(masks[r][i, j // 32]) >> (j % 32)) & 1
        want = ref.attention(q[r, :k + 1].double().numpy(), K, V, see, scale)
        # the weights: 2^-11 each and 2^-22 of the exponential; an exponent is off by 2^-23 of a distance
        # that counts (below 2^6) in a part, and equal scores have equal weights
        tol = 2.0 ** -8 * np.abs(want) + np.abs(V).max() * (2.0 ** -9 + (L + 16) * 2.0 ** -22)
        assert (np.abs(O[r, :k + 1] - want) <= tol).all()
