"""Attention with a sliding window and sinks over the paged 4-bit cache
against the formula in 64 bits: single tokens, draft trees, chains and packed
rows."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from speculative_decoding_draft_06_gb300 import dartree as dtl
from speculative_decoding_draft_06_gb300 import inputs as I
from tests import cache_ref as ref
from tests.test_gpu_cache import cu, host
from tests.test_gpu_cache_attention import filled, tolerance
from tests.test_gpu_verify import ancestor_mask

pytestmark = pytest.mark.gpu


def bits_of(mask, n):
    return np.array([[(int(mask[i, j // 32]) >> (j % 32)) & 1 for j in range(n)] for i in range(n)], bool).reshape(n, n)


def visible(base, rows, window, sinks, tree=None):
    """[rows, base + rows]: what the rows see; row 0 at position base, the
    others a chain or (``tree`` [rows - 1, rows - 1]) its nodes."""
    L = base + rows
    q = base + np.arange(rows)
    k = np.arange(L)
    see = k[None] <= q[:, None]
    if tree is not None:
        depth = np.concatenate([[0], tree.sum(1)]).astype(int)
        q = base + depth
        k = np.concatenate([np.arange(base + 1), base + depth[1:]])
        see = np.zeros((rows, L), bool)
        see[:, :base + 1] = True
        see[1:, base + 1:] = tree
    if window is None:
        return see
    return see & ((k[None] < sinks) | (q[:, None] - k[None] < window))


def check_request(O, q, K, V, see, scale):
    want = ref.attention(q, K, V, see, scale)
    err = np.abs(O - want)
    tol = tolerance(want, q, K, V, scale)
    assert (err <= tol).all(), (float((err - tol).max()), float((err / tol).max()))


def let_go(table, lens, base_of, P, window, sinks):
    """The table without the pages that a window has left behind."""
    t = table.copy()
    if window is not None:
        for r in range(len(lens)):
            s = np.arange(t.shape[1])
            t[r, (s * P >= sinks) & (s * P + P - 1 <= base_of[r] - window)] = -1
    return t


SINGLE = [  # R, Hq, Hkv, dh, P, window, sinks, lens
    (1, 8, 8, 128, 64, 1, 0, [1]), (1, 32, 8, 128, 64, 512, 4, [1000]), (3, 8, 2, 64, 16, 16, 1, [0, 17, 63]),
    (4, 12, 4, 128, 32, 64, 0, [64, 65, 127, 128]), (5, 5, 1, 128, 128, 63, 130, [1, 0, 129, 300, 1]),
    (2, 16, 1, 64, 64, 65, 100, [2000, 31]), (1, 32, 1, 128, 16, 2, 3, [333]), (2, 40, 2, 64, 128, None, 0, [500, 257]),
    (6, 4, 4, 64, 32, 100, 4, [33, -1, 700, 1, 95, 96]), (1, 7, 7, 128, 16, 4000, 4, [4500]),
    (40, 8, 2, 128, 64, 90, 4, list(range(0, 400, 10))), (3, 8, 2, 128, 16, 1 << 30, 5, [100, 1, 40]),
    (2, 8, 2, 128, 64, 5, 1 << 30, [700, 77]), (4, 8, 8, 64, 64, 3000, 64, [5000, 4097, 2900, 64]),
]


@pytest.mark.parametrize("case", range(len(SINGLE)))
def test_single_tokens(case):
    R, Hq, Hkv, dh, P, window, sinks, lens = SINGLE[case]
    g = np.random.default_rng(4000 + case)
    lens = np.array(lens)
    cache, table, vals = filled(g, lens, 0, P, Hkv, dh)
    table = let_go(table, lens, lens - 1, P, window, sinks)
    q = torch.from_numpy(g.standard_normal((R, 1, Hq, dh)) * 3).to(torch.bfloat16)
    for bound in (int(lens.max()), int(lens.max()) * 3 + 70):       # (other key splits)
        out = torch.full((R, 1, Hq, dh), 5.0, dtype=torch.bfloat16, device="cuda")
        cache.window_attention(0, q.cuda(), cu(table), cu(lens), window=window, sinks=sinks, max_len=bound, out=out)
        cache.check()
        O = host(out.double())
        for r, (K, V) in enumerate(vals):
            n = int(lens[r])
            if n < 0:
                assert (O[r] == 5.0).all()
            elif n == 0:
                assert (O[r] == 0.0).all()
            else:
                see = visible(n - 1, 1, window, sinks)
                check_request(O[r], q[r].double().numpy(), K[:n], V[:n], see, dh ** -0.5)


TREES = [  # R, B, Hq, Hkv, dh, P, window, sinks, lens
    (1, 1, 8, 8, 128, 64, 1, 0, [1]), (1, 3, 16, 4, 128, 64, 2, 1, [100]), (2, 7, 4, 2, 64, 16, 3, 2, [5, 61]),
    (1, 33, 8, 2, 128, 32, 20, 0, [63]), (3, 16, 6, 2, 64, 128, 40, 150, [1, 200, 9]),
    (2, 64, 8, 8, 128, 16, 64, 4, [130, 64]), (1, 130, 32, 8, 128, 64, 300, 4, [700]),
    (2, 40, 5, 1, 64, 64, None, 0, [1000, 3]), (1, 256, 16, 4, 128, 128, 7, 0, [64]),
    (4, 20, 16, 2, 128, 64, 100, 1, [50, -1, 333, 128]), (1, 128, 32, 8, 128, 64, 1024, 4, [2600]),
    (1, 1024, 4, 2, 64, 32, 5, 12, [10]), (2, 65, 64, 1, 128, 16, 33, 0, [257, 90]), (2, 9, 4, 2, 128, 16, 4, 3, [0, 2]),
]


@pytest.mark.parametrize("case", range(len(TREES)))
def test_trees(case):
    """Windows shorter than a tree is deep, sinks among its nodes, empty
    prefixes."""
    R, B, Hq, Hkv, dh, P, window, sinks, lens = TREES[case]
    g = np.random.default_rng(5000 + case)
    lens = np.array(lens)
    n = np.array([B] + [int(g.integers(0, B + 1)) for _ in range(R - 1)])
    if case % 2:  # half of the cases: trees that are deep
        parents = [np.array([max(-1, i - 1 - int(g.integers(0, 2))) for i in range(B)]) for _ in n]
    else:
        parents = [I.random_tree(g, B, max(1, int(k)))["parent"] for k in n]
    masks = np.stack([ancestor_mask(t, int(k), B) for t, k in zip(parents, n)])
    cache, table, vals = filled(g, lens, n, P, Hkv, dh)
    table = let_go(table, lens, lens - 1, P, window, sinks)
    q = torch.from_numpy(g.standard_normal((R, B + 1, Hq, dh)) * 2).to(torch.bfloat16)
    out = torch.full((R, B + 1, Hq, dh), 5.0, dtype=torch.bfloat16, device="cuda")
    top = int((np.maximum(lens, 0) + n).max())
    cache.window_attention(0, q.cuda(), cu(table), cu(lens), mask=torch.from_numpy(masks.view(np.int32)).cuda(),
                           n_nodes=cu(n), max_len=top, window=window, sinks=sinks, out=out)
    cache.check()
    O = host(out.double())
    for r, (K, V) in enumerate(vals):
        L, k = int(lens[r]), int(n[r])
        assert (O[r, (k + 1 if L >= 0 else 0):] == 5.0).all()
        if L < 0:
            continue
        see = visible(L - 1, k + 1, window, sinks, bits_of(masks[r], k))
        check_request(O[r, :k + 1], q[r, :k + 1].double().numpy(), K[:L + k], V[:L + k], see, dh ** -0.5)


CHAINS = [  # R, rows, Hq, Hkv, dh, P, window, sinks, lens (before row 0)
    (1, 2, 8, 8, 128, 64, 1, 0, [0]), (2, 4, 4, 1, 64, 16, 3, 2, [5, 0]), (3, 16, 8, 8, 128, 32, None, 0, [0, 9, 64]),
    (1, 17, 8, 8, 128, 64, 7, 0, [100]), (2, 131, 4, 2, 64, 64, 50, 4, [0, 63]), (1, 700, 8, 2, 128, 64, 129, 4, [0]),
    (2, 333, 6, 2, 128, 16, 64, 0, [130, 1]), (1, 1500, 3, 3, 64, 128, 200, 33, [77]), (1, 600, 4, 2, 128, 64, None, 0, [500]),
    (1, 1030, 1, 1, 128, 32, 1, 1, [0]), (4, 70, 10, 2, 64, 16, 31, 64, [0, -1, 2000, 16]), (1, 129, 1, 1, 64, 64, 40, 0, [3]),
]


@pytest.mark.parametrize("packed", [False, True])
@pytest.mark.parametrize("case", range(len(CHAINS)))
def test_chains(case, packed):
    """Prompts and drafted chains: rows in the order of their positions, padded
    (with fewer rows in some requests) and packed."""
    R, rows, Hq, Hkv, dh, P, window, sinks, lens = CHAINS[case]
    g = np.random.default_rng(6000 + case)
    lens = np.array(lens)
    n = np.array([rows] + [int(g.integers(1, rows + 1)) for _ in range(R - 1)])
    cache, table, vals = filled(g, lens, n, P, Hkv, dh)
    table = let_go(table, lens, lens, P, window, sinks)
    q = torch.from_numpy(g.standard_normal((R, rows, Hq, dh)) * 2).to(torch.bfloat16)
    top = int((np.maximum(lens, 0) + n).max())
    more = dict(max_len=top, window=window, sinks=sinks, offset=0)
    if packed:
        start = np.concatenate([[0], np.cumsum(n)])
        Q = torch.cat([q[r, :n[r]] for r in range(R)] + [q[0, :1]]).cuda()      # a row that belongs to nobody
        out = torch.full(Q.shape, 5.0, dtype=torch.bfloat16, device="cuda")
        cache.window_attention(0, Q, cu(table), cu(lens), start=cu(start), max_rows=rows, out=out, **more)
        new = cache.window_attention(0, Q, cu(table), cu(lens), start=cu(start), max_rows=rows, **more)
        O = host(out.double())
        got = [O[start[r]:start[r + 1]] for r in range(R)]
        rest = [O[start[R]:]]
    else:
        out = torch.full(q.shape, 5.0, dtype=torch.bfloat16, device="cuda")
        cache.window_attention(0, q.cuda(), cu(table), cu(lens), n_nodes=cu(n - 1), out=out, **more)
        new = cache.window_attention(0, q.cuda(), cu(table), cu(lens), n_nodes=cu(n - 1), **more)
        O = host(out.double())
        got = [O[r, :n[r]] for r in range(R)]
        rest = [O[r, n[r]:] for r in range(R)]
    cache.check()
    assert all((x == 5.0).all() for x in rest)
    live = np.ones(O.shape[:-2], bool)
    for r, (K, V) in enumerate(vals):
        L, k = int(lens[r]), int(n[r])
        if L < 0:
            assert (got[r] == 5.0).all()
        else:
            check_request(got[r], q[r, :k].double().numpy(), K[:L + k], V[:L + k], visible(L, k, window, sinks), dh ** -0.5)
    # a new output: the same rows, zeros in those that nobody has
    N = host(new.double())
    live = (O != 5.0).any((-1, -2))
    assert np.array_equal(N[live], O[live]) and not N[~live].any()


def test_no_window_is_the_plain_attention():
    """Without a window a tree's rows are those of `attention`, bit for bit."""
    g = np.random.default_rng(3)
    R, B, Hq, Hkv, dh, P = 2, 40, 8, 2, 128, 64
    lens, n = np.array([300, 0]), np.array([40, 17])
    masks = np.stack([ancestor_mask(I.random_tree(g, B, int(k))["parent"], int(k), B) for k in n])
    cache, table, _ = filled(g, lens, n, P, Hkv, dh)
    q = torch.from_numpy(g.standard_normal((R, B + 1, Hq, dh))).to(torch.bfloat16).cuda()
    m = torch.from_numpy(masks.view(np.int32)).cuda()
    a = cache.attention(0, q, cu(table), cu(lens), mask=m, n_nodes=cu(n), max_len=340)
    b = cache.window_attention(0, q, cu(table), cu(lens), mask=m, n_nodes=cu(n), max_len=340)
    cache.check()
    assert torch.equal(a, b)


@pytest.mark.parametrize("rows", [1, 40])
def test_missing_pages(rows):
    """A page that is missing inside the window, or has a bad number, is not
    seen and flagged; outside it is not looked at."""
    g = np.random.default_rng(8)
    Hq, Hkv, dh, P, window, sinks = 4, 2, 64, 16, 70, 4
    lens = np.array([400, 400, 400])
    cache, table, vals = filled(g, lens, rows, P, Hkv, dh)
    table[:, 3:12] = -1                       # far behind the window (from token 331 on)
    table[0, 5] = 1 << 20
    q = torch.from_numpy(g.standard_normal((3, rows, Hq, dh))).to(torch.bfloat16)
    run = lambda: host(cache.window_attention(0, q.cuda(), cu(table), cu(lens), max_len=400 + rows, window=window,  # noqa: E731
                                              sinks=sinks, offset=0).double())
    O = run()
    cache.check()
    table[1, 22] = 1 << 20                    # tokens 352 .. 367
    table[2, 0] = -1                          # the sinks
    B = run()
    with pytest.raises(dtl.DartreeError):
        cache.check()
    assert np.array_equal(O[0], B[0])
    for r, gone in ((1, slice(352, 368)), (2, slice(0, 16))):
        K, V = vals[r]
        see = visible(400, rows, window, sinks)
        see[:, gone] = False
        check_request(B[r], q[r].double().numpy(), K[:400 + rows], V[:400 + rows], see, dh ** -0.5)


def test_bad_packed_rows_are_skipped_and_flagged():
    g = np.random.default_rng(9)
    lens = np.array([20, 30, 40])
    cache, table, vals = filled(g, lens, 4, 16, 2, 64)
    q = torch.from_numpy(g.standard_normal((6, 4, 64))).to(torch.bfloat16)
    for start in ([0, 2, 4, 7], [-1, 2, 4, 6], [0, 2, 6, 4], [0, 5, 5, 6]):
        out = torch.full((6, 4, 64), 5.0, dtype=torch.bfloat16, device="cuda")
        cache.window_attention(0, q.cuda(), cu(table), cu(lens), start=cu(start), max_rows=4, max_len=44, window=9,
                               offset=0, out=out)
        with pytest.raises(dtl.DartreeError):
            cache.check()
        O = host(out.double())
        for r in range(3):
            a, b = start[r], start[r + 1]
            if 0 <= a < b <= 6 and b - a <= 4:
                L, k = int(lens[r]), b - a
                check_request(O[a:b], q[a:b].double().numpy(), vals[r][0][:L + k], vals[r][1][:L + k],
                              visible(L, k, 9, 0), 64 ** -0.5)


def test_strides_scale_layer_and_graph():
    """Packed queries sliced from a fused projection, a later layer, scale
    exponents; a captured call follows lens, start and the table."""
    g = np.random.default_rng(10)
    Hq, Hkv, dh, P = 8, 2, 128, 64
    lens = np.array([200, 77])
    cache, table, vals = filled(g, lens, 60, P, Hkv, dh, ks=2.0 ** 7, vs=2.0 ** -9, layers=2)
    fused = torch.from_numpy(g.standard_normal((40, (Hq + 2 * Hkv) * dh)) * 2.0 ** -8).to(torch.bfloat16).cuda()
    Q = fused[:, :Hq * dh].view(40, Hq, dh)
    t, ln, start = cu(table), cu(lens), cu([0, 25, 40])
    out = torch.zeros(40, Hq, dh, dtype=torch.bfloat16, device="cuda")
    call = lambda: cache.window_attention(1, Q, t, ln, start=start, max_rows=30, max_len=240, window=50, sinks=3,  # noqa: E731
                                          offset=0, scale=0.7, out=out)
    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for L, s in (([200, 77], [0, 25, 40]), ([180, 90], [0, 11, 37])):
        ln.copy_(cu(L))
        start.copy_(cu(s))
        out.fill_(0)
        graph.replay()
        cache.check()
        O = host(out.double())
        for r in range(2):
            k = s[r + 1] - s[r]
            check_request(O[s[r]:s[r + 1]], host(Q.double())[s[r]:s[r + 1]], vals[r][0][:L[r] + k], vals[r][1][:L[r] + k],
                          visible(L[r], k, 50, 3), 0.7)


def test_refusals():
    cache = dtl.KVCache(1, 8, page_tokens=16, Hkv=2, dh=64)
    t, ln = cu(np.zeros((2, 4), np.int32)), cu([3, 4])
    q = torch.zeros(2, 3, 4, 64, dtype=torch.bfloat16, device="cuda")
    p = torch.zeros(6, 4, 64, dtype=torch.bfloat16, device="cuda")
    call = lambda Q, **k: cache.window_attention(0, Q, t, ln, max_len=9, **k)  # noqa: E731
    for Q, k in ((q, dict(window=0)), (q.float(), {}), (p, {}), (q, dict(start=cu([0, 1, 2]))),
                 (p, dict(start=cu([0, 1, 2]))), (p, dict(start=cu([0, 1]), max_rows=2)),
                 (p, dict(start=cu([0, 1, 2]), max_rows=2, n_nodes=cu([1, 1]))), (q, dict(n_nodes=cu([1]))),
                 (q[:, :, :3], {}), (q, dict(out=q[:1])), (q, dict(sinks=-1)), (q, dict(scale=-1.0)),
                 (q, dict(mask=cu([0, 0]))), (q.transpose(1, 2).contiguous().transpose(1, 2), {}),
                 (q, dict(work=torch.zeros(4, 4, device="cuda").t()))):
        with pytest.raises((TypeError, ValueError, dtl.DartreeError)):
            call(Q, **k)
    big = torch.zeros(2, 1026, 4, 64, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(dtl.DartreeError):
        call(big, mask=cu(np.zeros((2, 1025, 33), np.int32)))
    call(q)
    cache.err.zero_()
