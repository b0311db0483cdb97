"""Attention over the cache where a CTA's warps work through many key tiles:
refilled stages, one split with all keys, splits that join through the
workspace by one warp and by eight, leftover rows of trees.  The sequences
share a set of pages in random order, so that every tile differs from its
neighbours and the 64-bit reference stays small."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from speculative_decoding_draft_06_gb300 import dartree as dtl
from speculative_decoding_draft_06_gb300 import inputs as I
from tests import cache_ref as ref
from tests.test_gpu_cache import cu, host
from tests.test_gpu_verify import ancestor_mask

pytestmark = pytest.mark.gpu


def pages_of(g, N, P, Hkv, dh):
    """A cache of N pages, and their keys and values [N, P, Hkv, dh] in fp64."""
    cache = dtl.KVCache(1, N + 1, page_tokens=P, Hkv=Hkv, dh=dh)
    cache.pool.fill_(0x7F)
    out = []
    x = [torch.from_numpy(g.standard_normal((1, N * P, Hkv, dh))).to(torch.bfloat16) for _ in range(2)]
    cache.append(0, x[0].cuda(), x[1].cuda(), cu(np.arange(N)[None]), cu([0]))
    for y in x:
        out.append(ref.values(*ref.quantise(y[0].double().numpy())).reshape(N, P, Hkv, dh))
    cache.check()
    return cache, out[0], out[1]


def check_request(O, q, K, V, see, scale, keys):
    """O, q [n, Hq, dh] against the formula over K, V [L, Hkv, dh].  The output is
    rounded to bf16 (2^-8), the weights to fp16 (2^-11 of each; 2^-25 of the
    scaled range below 2^-14 of it, the range's unit being at most 2^6 below
    the largest weight); a score's sum is off by (dh + 8) 2^-23 sum|q k|, in a
    weight and in the normaliser.  A warp sums `keys` keys, and some 80 shares
    are added behind it, by 2^-23 each at most.  All but the first are
    relative to sum w |v|."""
    want, mass = ref.attention(q, K, V, see, scale), ref.attention(q, K, np.abs(V), see, scale)
    s = scale * np.abs(q).max() * np.abs(K).sum(-1).max(initial=0.0)
    d = (K.shape[2] + 8) * 2.0 ** -23 * s
    tol = 2.0 ** -8 * np.abs(want) + mass * (2.0 ** -10 + 2 * d + (keys + 80) * 2.0 ** -23) + K.shape[0] * 2.0 ** -31 * 8 + 1e-30
    err = np.abs(O - want)
    assert (err <= tol).all(), (float((err - tol).max()), float((err / tol).max()))


CASES = [  # R, Hq, Hkv, dh, P, lengths (from, to), long ones, B, bound beyond them
    (58, 32, 8, 128, 64, (1500, 2500), (), 0, 0),        # two splits, five tiles a warp, through the workspace
    (230, 16, 2, 64, 16, (600, 1200), (), 0, 0),        # one split
    (120, 64, 4, 128, 128, (900, 1500), (), 0, 0),       # one, sixteen rows
    (58, 96, 8, 64, 32, (700, 1300), (1, 64), 0, 0),
    (58, 24, 8, 128, 16, (1000, 1700), (0, 63, 65), 0, 0),
    (64, 32, 8, 128, 64, (1, 700), (13000, 4096, 4097, 8192, 12288), 0, 0),  # seven splits, joined by a warp a row
    (64, 64, 4, 64, 16, (1, 500), (13001, 9000), 0, 0),
    (58, 32, 8, 128, 128, (300, 2500), (), 0, 17500),    # a loose bound: nine splits, most without keys
    (1, 32, 8, 128, 64, (41003, 41003), (), 0, 0),       # 53 splits, three tiles a warp, joined by eight warps
    (1, 128, 8, 64, 128, (40500, 40500), (), 0, 0),
    (2, 8, 1, 128, 16, (70001, 70001), (33333,), 0, 0),
    (64, 32, 8, 128, 64, (1500, 2300), (1,), 3, 0),      # small trees: nodes behind many tiles
    (60, 16, 8, 64, 16, (1000, 1500), (0, 700), 7, 0),
    (2, 32, 8, 128, 64, (6000, 6100), (), 128, 0),       # four rows behind whole tiles: three tiles a warp
    (30, 32, 8, 128, 32, (2500, 3000), (5,), 32, 0),     # six
    (12, 8, 8, 64, 16, (3000, 4000), (), 130, 0),
    (8, 32, 8, 128, 64, (4000, 4100), (100,), 0, 0),     # six splits in a cluster, three tiles a warp
    (19, 64, 8, 64, 32, (1000, 1700), (0,), 0, 0),       # three
]


@pytest.mark.parametrize("case", range(len(CASES)))
def test_many_tiles(case):
    R, Hq, Hkv, dh, P, (lo, hi), long, B, loose = CASES[case]
    g = np.random.default_rng(4000 + case)
    lens = g.integers(lo, hi + 1, R)
    lens[g.permutation(R)[:len(long)]] = long
    n = np.full(R, B)
    if B:
        n[1:] = g.integers(max(0, B - 3), B + 1, R - 1)
    N = max(20, 2000 // P)
    cache, Kp, Vp = pages_of(g, N, P, Hkv, dh)
    held = -(-(lens + n) // P)
    table = np.full((R, int(held.max()) + 1), -1)
    for r in range(R):
        table[r, :held[r]] = g.integers(0, N, held[r])
    masks = np.stack([ancestor_mask(I.random_tree(g, max(B, 1), max(1, int(k)))["parent"], int(k), max(B, 1)) for k in n])
    q = torch.from_numpy(g.standard_normal((R, B + 1, Hq, dh)) * 3).to(torch.bfloat16)
    kw = dict(mask=torch.from_numpy(masks.view(np.int32)).cuda(), n_nodes=cu(n)) if B else {}
    most = int((lens + n).max()) + loose
    out = cache.attention(0, q.cuda(), cu(table), cu(lens), max_len=most, **kw)
    again = cache.attention(0, q.cuda(), cu(table), cu(lens), max_len=most, **kw)
    cache.check()
    assert torch.equal(out, again)
    O, q = host(out.double()), q.double().numpy()
    for r in range(R):
        L, k = int(lens[r]), int(n[r])
        K, V = (x[table[r, :held[r]]].reshape(-1, Hkv, dh)[:L + k] for x in (Kp, Vp))
        see = np.zeros((k + 1, L + k), bool)
        see[:, :L] = True
        bits = np.unpackbits(masks[r].view(np.uint8), axis=1, bitorder="little")
        see[1:, L:] = bits[:k, :k]
        check_request(O[r, :k + 1], q[r, :k + 1], K, V, see, dh ** -0.5, L + k)


@pytest.mark.parametrize("R,Hq,Hkv,dh,P", [(58, 32, 8, 128, 64), (58, 16, 8, 64, 16), (58, 8, 8, 128, 32),
                                           (230, 32, 2, 64, 128), (2, 8, 2, 128, 64)])
def test_missing_pages_behind_the_first_stages(R, Hq, Hkv, dh, P):
    """Pages that are not there in tiles that refill a stage: not seen, and what
    the stage held before is not seen either."""
    g = np.random.default_rng(R + P)
    lens = g.integers(1200, 2000, R) if R > 2 else np.array([30000, 20000])
    N = max(20, 2000 // P)
    cache, Kp, Vp = pages_of(g, N, P, Hkv, dh)
    held = -(-lens // P)
    table = np.full((R, int(held.max())), -1)
    for r in range(R):
        table[r, :held[r]] = g.integers(0, N, held[r])
        gone = g.random(held[r]) < 0.2
        gone[:512 // P] = False
        table[r, :held[r]][gone] = g.choice([-1, N + 1, 2 ** 30], int(gone.sum()))
    q = torch.from_numpy(g.standard_normal((R, 1, Hq, dh)) * 3).to(torch.bfloat16)
    out = cache.attention(0, q.cuda(), cu(table), cu(lens), max_len=int(lens.max()))
    with pytest.raises(dtl.DartreeError):
        cache.check()
    O, q = host(out.double()), q.double().numpy()
    for r in range(R):
        row = table[r, :held[r]]
        there = (row >= 0) & (row < N)
        K, V = (x[np.where(there, row, 0)].reshape(-1, Hkv, dh)[:lens[r]] for x in (Kp, Vp))
        see = np.repeat(there, P)[None, :lens[r]]
        check_request(O[r], q[r], K, V, see, dh ** -0.5, int(lens[r]))
