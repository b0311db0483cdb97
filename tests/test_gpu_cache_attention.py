"""Attention over the paged 4-bit cache against the formula in 64 bits, and
the verification step that uses the cache, its page operations and the
sampling together."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import oracle
from speculative_decoding_draft_06_gb300 import dartree as dtl
from speculative_decoding_draft_06_gb300 import inputs as I
from tests import cache_ref as ref
from tests import gpu_util as gu
from tests.test_gpu_cache import cu, host, tables
from tests.test_gpu_verify import ancestor_mask

pytestmark = pytest.mark.gpu


def tolerance(O, q, K, V, scale):
    """Rounding of one row set against the 64-bit result.  The output is
    rounded to bf16 (2^-8 of the value).  The weights are rounded to fp16
    (2^-11 of each; below 2^-14 of the scaled range, 2^-25 of it, the range's
    unit being at most 2^6 below the largest weight), and come from scores
    whose dh-term fp32 sums are off by at most dh 2^-23 sum|q k|: a factor
    e^d on each, in the sum and its normaliser.  Products with the values
    are summed in fp32 over L keys."""
    L, dh = K.shape[0], K.shape[2]
    vmax = np.abs(V).max(initial=0.0)
    s = scale * np.abs(q).max(initial=0.0) * np.abs(K).sum(-1).max(initial=0.0)
    d = (dh + 8) * 2.0 ** -23 * s
    return 2.0 ** -8 * np.abs(O) + vmax * (2.0 ** -10 + L * 2.0 ** -31 + 2 * d + (L + 16) * 2.0 ** -22) + 1e-30


def filled(g, lens, n, P, Hkv, dh, ks=1.0, vs=1.0, layers=1, extra_pages=2):
    """A cache whose rows hold lens + n tokens each (everything else is the
    byte 0x7F: an e4m3 NaN), and the tokens' values in fp64."""
    R = len(lens)
    total = np.maximum(lens, 0) + n
    table, refs = tables(g, -(-total // P), int((-(-total // P)).sum()) + extra_pages, max(1, int(-(-total.max() // P))) + 1)
    cache = dtl.KVCache(layers, len(refs), page_tokens=P, Hkv=Hkv, dh=dh, k_scale=ks, v_scale=vs, refs=cu(refs))
    cache.pool.fill_(0x7F)
    vals = []
    for r in range(R):
        x = torch.from_numpy(g.standard_normal((2, 1, max(1, total[r]), Hkv, dh)) * [[[[[1.0]]]], [[[[2.0]]]]]).to(torch.bfloat16)
        x = x * torch.tensor([ks, vs], dtype=torch.bfloat16).view(2, 1, 1, 1, 1)
        if total[r]:
            cache.append(layers - 1, x[0].cuda(), x[1].cuda(), cu(table[r:r + 1]), cu([0]))
        vals.append(tuple(ref.values(*ref.quantise(x[i, 0, :total[r]].double().numpy(), u), u)
                          for i, u in ((0, ks), (1, vs))))
    cache.check()
    return cache, table, vals


def check_rows(O, q, lens, n, masks, vals, scale):
    """Every live row of O [R, B+1, Hq, dh] against the formula."""
    for r, (K, V) in enumerate(vals):
        if lens[r] < 0:
            continue
        L, k = int(lens[r]), int(n[r])
        see = np.zeros((k + 1, L + k), bool)
        see[:, :L] = True
        for i in range(k):
            for j in range(k):
                see[i + 1, L + j] = (int(masks[r][i, j // 32]) >> (j % 32)) & 1
        want = ref.attention(q[r, :k + 1], K[:L + k], V[:L + k], see, scale)
        err = np.abs(O[r, :k + 1] - want)
        tol = tolerance(want, q[r, :k + 1], K[:L + k], V[:L + k], scale)
        assert (err <= tol).all(), (r, float((err - tol).max()), float((err / tol).max()))


SINGLE = [  # R, Hq, Hkv, dh, P, lens
    (1, 8, 8, 128, 64, [1]), (1, 32, 8, 128, 64, [1000]), (3, 8, 2, 64, 16, [0, 17, 63]),
    (4, 12, 4, 128, 32, [64, 65, 127, 128]), (5, 5, 1, 128, 128, [1, 0, 129, 300, 1]), (2, 16, 1, 64, 64, [2000, 31]),
    (1, 32, 1, 128, 16, [333]), (2, 40, 2, 64, 128, [500, 257]), (6, 4, 4, 64, 32, [33, -1, 700, 1, 95, 96]),
    (1, 7, 7, 128, 16, [4500]), (40, 8, 2, 128, 64, list(range(0, 400, 10))),
]


@pytest.mark.parametrize("case", range(len(SINGLE)))
def test_single_tokens(case):
    R, Hq, Hkv, dh, P, lens = SINGLE[case]
    g = np.random.default_rng(1000 + case)
    lens = np.array(lens)
    cache, table, vals = filled(g, lens, 0, P, Hkv, dh)
    q = torch.from_numpy(g.standard_normal((R, 1, Hq, dh)) * 3).to(torch.bfloat16)
    out = torch.full((R, 1, Hq, dh), 5.0, dtype=torch.bfloat16, device="cuda")
    cache.attention(0, q.cuda(), cu(table), cu(lens), max_len=int(lens.max()), out=out)
    cache.check()
    O = host(out.double())
    check_rows(O, q.double().numpy(), lens, [0] * R, None, vals, dh ** -0.5)
    for r in range(R):
        assert lens[r] >= 0 or (O[r] == 5.0).all()       # a skipped row
        assert lens[r] != 0 or (O[r] == 0.0).all()       # nothing to see
    # a looser bound of the lengths: other key splits, the same values up to rounding
    loose = cache.attention(0, q.cuda(), cu(table), cu(lens), max_len=int(lens.max()) * 3 + 70, out=out.clone())
    cache.check()
    check_rows(host(loose.double()), q.double().numpy(), lens, [0] * R, None, vals, dh ** -0.5)


TREES = [  # R, B, Hq, Hkv, dh, P, lens
    (1, 1, 8, 8, 128, 64, [0]), (1, 3, 16, 4, 128, 64, [100]), (2, 7, 4, 2, 64, 16, [5, 61]),
    (1, 33, 8, 2, 128, 32, [63]), (3, 16, 6, 2, 64, 128, [1, 200, 0]), (2, 64, 8, 8, 128, 16, [130, 64]),
    (1, 130, 32, 8, 128, 64, [700]), (2, 40, 5, 1, 64, 64, [1000, 3]), (1, 256, 16, 4, 128, 128, [64]),
    (4, 20, 16, 2, 128, 64, [50, -1, 333, 128]), (1, 128, 32, 8, 128, 64, [3000]), (1, 1024, 4, 2, 64, 32, [10]),
    (2, 65, 64, 1, 128, 16, [257, 90]),
]


@pytest.mark.parametrize("case", range(len(TREES)))
def test_trees(case):
    """Trees smaller than B, rows behind them left as they were, prefixes
    that end inside a page and a tile, empty prefixes (the root sees
    nothing)."""
    R, B, Hq, Hkv, dh, P, lens = TREES[case]
    g = np.random.default_rng(2000 + case)
    lens = np.array(lens)
    n = np.array([B] + [int(g.integers(0, B + 1)) for _ in range(R - 1)])
    trees = [I.random_tree(g, B, max(1, int(k))) for k in n]
    masks = np.stack([ancestor_mask(t["parent"], int(k), B) for t, k in zip(trees, n)])
    cache, table, vals = filled(g, lens, n, P, Hkv, dh)
    q = torch.from_numpy(g.standard_normal((R, B + 1, Hq, dh)) * 2).to(torch.bfloat16)
    out = torch.full((R, B + 1, Hq, dh), 5.0, dtype=torch.bfloat16, device="cuda")
    top = int((np.maximum(lens, 0) + n).max())
    cache.attention(0, q.cuda(), cu(table), cu(lens), mask=torch.from_numpy(masks.view(np.int32)).cuda(),
                    n_nodes=cu(n), max_len=top, out=out)
    cache.check()
    O = host(out.double())
    check_rows(O, q.double().numpy(), lens, n, masks, vals, dh ** -0.5)
    for r in range(R):
        assert (O[r, (n[r] + 1 if lens[r] >= 0 else 0):] == 5.0).all()
        assert lens[r] != 0 or (O[r, 0] == 0.0).all()


@pytest.mark.parametrize("B", [0, 5, 40])
def test_scales_layers_strides_and_large_scores(B):
    """Scale exponents, a later layer, queries sliced from a fused projection,
    a scale that makes the softmax nearly one-hot, queries of very different
    sizes (a row is scaled by its own power of two)."""
    g = np.random.default_rng(31 + B)
    R, Hq, Hkv, dh, P = 2, 8, 2, 128, 64
    lens = np.array([200, 77])
    n = np.array([B, max(0, B - 3)])
    masks = np.stack([ancestor_mask(I.random_tree(g, max(B, 1), max(1, int(k)))["parent"], int(k), max(B, 1)) for k in n])
    cache, table, vals = filled(g, lens, n, P, Hkv, dh, ks=2.0 ** 7, vs=2.0 ** -9, layers=3)
    fused = torch.from_numpy(g.standard_normal((R, B + 1, Hq * dh + 2 * Hkv * dh))
                             * 2.0 ** g.integers(-30, -4, (R, B + 1, 1))).to(torch.bfloat16).cuda()
    Q = fused[:, :, :Hq * dh].view(R, B + 1, Hq, dh)
    assert not Q.is_contiguous()
    m = torch.from_numpy(masks.view(np.int32)).cuda() if B else None
    for scale in (0.5, 20.0):
        out = cache.attention(2, Q, cu(table), cu(lens), mask=m, n_nodes=cu(n), max_len=300, scale=scale)
        cache.check()
        check_rows(host(out.double()), host(Q.double()), lens, n, masks, vals, scale)


def test_bad_pages_are_not_seen_and_flagged():
    """A page that is missing or does not exist: its tokens are not seen; a
    length beyond max_len: the tokens behind it are not."""
    g = np.random.default_rng(5)
    lens = np.array([150, 150, 150])
    cache, table, vals = filled(g, lens, 0, 32, 2, 64)
    table[1, 2] = len(host(cache.refs))                  # out of range
    table[2, 3] = -1
    q = torch.from_numpy(g.standard_normal((3, 1, 4, 64))).to(torch.bfloat16)
    out = cache.attention(0, q.cuda(), cu(table), cu(lens), max_len=150)
    with pytest.raises(dtl.DartreeError):
        cache.check()
    O = host(out.double())
    for r, hole in ((0, None), (1, 2), (2, 3)):
        K, V = vals[r]
        see = np.ones((1, 150), bool)
        if hole is not None:
            see[:, 32 * hole:32 * hole + 32] = False
        want = ref.attention(q[r].double().numpy(), K, V, see, 64 ** -0.5)
        assert (np.abs(O[r] - want) <= tolerance(want, q[r].double().numpy(), K, V, 64 ** -0.5)).all()
    out = cache.attention(0, q[:1].cuda(), cu(table[:1]), cu(lens[:1]), max_len=100)
    with pytest.raises(dtl.DartreeError):
        cache.check()
    want = ref.attention(q[0].double().numpy(), vals[0][0][:100], vals[0][1][:100], np.ones((1, 100), bool), 64 ** -0.5)
    assert (np.abs(host(out.double())[0] - want) <=
            tolerance(want, q[0].double().numpy(), *vals[0], 64 ** -0.5)).all()


def test_long_cache_in_many_splits():
    """A length that is shared over many CTAs; repeated calls are bit-equal."""
    g = np.random.default_rng(6)
    lens = np.array([20011, 3])
    cache, table, vals = filled(g, lens, 0, 128, 1, 128)
    q = torch.from_numpy(g.standard_normal((2, 1, 4, 128)) * 2).to(torch.bfloat16)
    a = cache.attention(0, q.cuda(), cu(table), cu(lens), max_len=20011)
    b = cache.attention(0, q.cuda(), cu(table), cu(lens), max_len=20011)
    cache.check()
    assert torch.equal(a, b)
    check_rows(host(a.double()), q.double().numpy(), lens, [0, 0], None, vals, 128 ** -0.5)


def test_captured_calls_and_other_streams():
    """Two graphs with workspaces of their own, replayed in turn after the
    lengths and the cache have changed, and a call on another stream."""
    g = np.random.default_rng(8)
    P, Hkv, dh, Hq = 64, 2, 128, 8
    lens = np.array([900, 400])
    cache, table, vals = filled(g, lens, 0, P, Hkv, dh)
    q = torch.from_numpy(g.standard_normal((2, 1, Hq, dh))).to(torch.bfloat16).cuda()
    t, ln = cu(table), cu(lens)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    eager = cache.attention(0, q, t, ln, max_len=1000, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    graphs, outs = [], []
    for _ in range(2):
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            outs.append(cache.attention(0, q, t, ln, max_len=1000))
        graphs.append(gr)
    for cut in (0, 333):
        ln.copy_(cu(np.maximum(lens - cut, 0)))
        for gr in graphs:
            gr.replay()
        torch.cuda.synchronize()
        assert torch.equal(outs[0], outs[1])
        check_rows(host(outs[0].double()), host(q.double()), np.maximum(lens - cut, 0), [0, 0], None, vals, dh ** -0.5)
        if cut == 0:
            assert torch.equal(outs[0], eager)
    cache.check()


def tree_call(g, lens, n, B, Hq, Hkv, dh, P):
    """A cache, queries and masks of trees of n nodes: what attention takes."""
    trees = [I.random_tree(g, B, max(1, int(k))) for k in n]
    masks = np.stack([ancestor_mask(t["parent"], int(k), B) for t, k in zip(trees, n)])
    cache, table, vals = filled(g, lens, n, P, Hkv, dh)
    q = torch.from_numpy(g.standard_normal((len(lens), B + 1, Hq, dh)) * 2).to(torch.bfloat16).cuda()
    return cache, table, vals, masks, torch.from_numpy(masks.view(np.int32)).cuda(), q


@pytest.mark.parametrize("Hq,Hkv,dh", [(8, 2, 128), (3, 1, 64), (8, 1, 128)])
def test_rows_behind_whole_tiles(Hq, Hkv, dh):
    """Trees whose rows end around multiples of 128, some with up to eight rows
    left over, of different lengths in one call and each alone without sizes."""
    g, gr, P, B = np.random.default_rng(Hq + dh), Hq // Hkv, 32, 170
    n = sorted({max(0, min(B, t * 128 // gr + d - 1)) for t in (1, 2, 4) for d in (-1, 0, 1, 2, 3, 5, 9)})
    lens = g.integers(0, 700, len(n))
    lens[::5] = 0
    n = np.array(n)
    cache, table, vals, masks, m, q = tree_call(g, lens, n, B, Hq, Hkv, dh, P)
    out = torch.full(q.shape, 5.0, dtype=torch.bfloat16, device="cuda")
    cache.attention(0, q, cu(table), cu(lens), mask=m, n_nodes=cu(n), max_len=int((lens + n).max()), out=out)
    cache.check()
    O = host(out.double())
    check_rows(O, host(q.double()), lens, n, masks, vals, dh ** -0.5)
    for r in range(len(n)):
        assert (O[r, n[r] + 1:] == 5.0).all()
        if n[r] > 0 and n[r] % 32 == 0:
            k = int(n[r])
            alone = cache.attention(0, q[r:r + 1, :k + 1].contiguous(), cu(table[r:r + 1]), cu(lens[r:r + 1]),
                                    mask=m[r:r + 1, :k, :k // 32].contiguous(), max_len=int(lens[r]) + k)
            check_rows(host(alone.double()), host(q[r:r + 1].double()), lens[r:r + 1], n[r:r + 1], masks[r:r + 1],
                       vals[r:r + 1], dh ** -0.5)
    cache.check()


@pytest.mark.parametrize("R", [255, 257, 300])
def test_trees_of_many_requests(R):
    g = np.random.default_rng(R)
    B, Hq, Hkv, dh, P = 5, 4, 1, 64, 16
    lens, n = g.integers(-1, 150, R), g.integers(0, B + 1, R)
    cache, table, vals, masks, m, q = tree_call(g, lens, n, B, Hq, Hkv, dh, P)
    out = cache.attention(0, q, cu(table), cu(lens), mask=m, n_nodes=cu(n), max_len=160)
    cache.check()
    check_rows(host(out.double()), host(q.double()), lens, n, masks, vals, dh ** -0.5)


def test_pages_behind_the_first_4_gb():
    """Attention of both kinds, commit and fork over far pages: the same bits
    as over near ones with the same bytes."""
    g = np.random.default_rng(21)
    Hkv, dh, P, Hq, B = 8, 128, 128, 16, 64
    cache = dtl.KVCache(2, 20000, page_tokens=P, Hkv=Hkv, dh=dh)       # 5.9 GB
    near, far = np.arange(6), np.array([19999, 14600, 19998, 16000, 15001, 18000])
    K = torch.randn(1, 6 * P, Hkv, dh, device="cuda").to(torch.bfloat16)
    for layer in range(2):
        cache.append(layer, K * (layer + 1), -K, cu(near[None]), cu([0]))
    cache.copy_pages(cu(near), cu(far))
    lens, n = np.array([650]), np.array([B])
    m = torch.from_numpy(ancestor_mask(I.random_tree(g, B, B)["parent"], B, B)[None].view(np.int32)).cuda()
    q = torch.randn(1, B + 1, Hq, dh, device="cuda").to(torch.bfloat16)
    for rows in (1, B + 1):
        kw = dict(mask=m, n_nodes=cu(n)) if rows > 1 else {}
        out = [cache.attention(1, q[:, :rows].contiguous(), cu(t[None]), cu(lens), max_len=720, **kw) for t in (near, far)]
        assert torch.equal(*out)
    nodes, length = cu([[3, 9, 40]]), cu([3])
    read = []
    for t in (near, far):
        ln = cu(lens)
        cache.commit(cu(t[None]), ln, nodes, length)
        assert host(ln).tolist() == [653]
        read.append(cache.read(1, cu(t[None]), cu([0]), 653))
    assert torch.equal(read[0][0], read[1][0]) and torch.equal(read[0][1], read[1][1])
    cache.refs[torch.from_numpy(far).cuda()] = 1
    cache.refs[:6] = 1
    table, ln = cu(np.stack([far, np.full(6, -1)])), cu([653, 0])
    assert host(cache.fork(table, ln, cu([0]), cu([1]))).tolist() == [1]
    k, v = cache.read(1, table[1:].contiguous(), cu([0]), 653)
    cache.check()
    assert torch.equal(k, read[0][0]) and torch.equal(v, read[0][1])


@pytest.mark.parametrize("B", [0, 40])
def test_a_graph_with_branches(B):
    """Calls behind an event of another stream, behind two streams at once and
    behind copies, in a captured graph: the same bits as one after the other."""
    g = np.random.default_rng(60 + B)
    Hkv, dh, Hq, P = 2, 128, 8, 64
    lens, n = np.array([700, 300]), np.array([B, B])
    cache, table, vals, masks, m, q = tree_call(g, lens, n, max(B, 1), Hq, Hkv, dh, P)
    q = q[:, :B + 1].contiguous()
    t, start, ln = cu(table), cu(lens), cu(lens)
    K = torch.randn(2, 2, Hkv, dh, device="cuda").to(torch.bfloat16)
    logits, u = torch.randn(2 * (B + 1), 500, device="cuda"), torch.rand(2 * (B + 1), device="cuda")
    nodes, length = cu([[0, 2], [1, 0]]), cu([2 if B else 0, 1 if B else 0])
    kw = dict(mask=m, n_nodes=cu(n)) if B else {}
    side = torch.cuda.Stream()

    def run(branch):
        ln.copy_(start)
        cache.append(0, K, -K, t, ln, offset=-2)
        if branch:
            side.wait_stream(torch.cuda.current_stream())
        s = side if branch else None
        a = cache.attention(0, q, t, ln, max_len=800, stream=s, **kw)
        k, v = cache.read(0, t, ln, 2, offset=-2)
        d = dtl.sample(logits, u, rows_per_req=B + 1)
        if branch:
            torch.cuda.current_stream().wait_stream(side)
        cache.commit(t, ln, nodes, length, extra=1)
        b = cache.attention(0, q, t, ln, max_len=800, **kw)
        return a, k, v, d["token"], d["prob"], ln.clone(), b

    pool = cache.pool.clone()
    want = run(False)
    torch.cuda.synchronize()
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        got = run(True)
    for _ in range(3):
        cache.pool.copy_(pool)
        gr.replay()
        torch.cuda.synchronize()
        for x, y in zip(got, want):  # (the last reads a token that nothing has written: NaN)
            assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))
        assert not torch.isnan(got[0]).any()


def test_trees_on_two_streams_and_in_graphs():
    """Two streams and two graphs, each call with its own workspace: the same
    bits as alone."""
    g = np.random.default_rng(12)
    lens, n = np.array([2500]), np.array([64])
    cache, table, vals, masks, m, q = tree_call(g, lens, n, 64, 16, 4, 128, 64)
    t, ln, nn = cu(table), cu(lens), cu(n)
    call = lambda s=None: cache.attention(0, q, t, ln, mask=m, n_nodes=nn, max_len=2564, stream=s)  # noqa: E731
    want = call()
    check_rows(host(want.double()), host(q.double()), lens, n, masks, vals, 128 ** -0.5)
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    outs = [call(s) for _ in range(20) for s in streams]
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) for o in outs)
    graphs, outs = [torch.cuda.CUDAGraph() for _ in range(2)], []
    for gr in graphs:
        with torch.cuda.graph(gr):
            outs.append(call())
    torch.cuda.synchronize()
    for _ in range(10):
        for s, gr in zip(streams, graphs):
            with torch.cuda.stream(s):
                gr.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) for o in outs)
    cache.check()


def test_verification_steps_over_the_cache():
    """Three steps of one layer, as a user runs them: build a tree, reserve
    pages, append the root's and the nodes' keys and values, attend, sample
    the target's tokens, accept, commit, let the surplus pages go -- and a
    fork that goes on from there.  The cache must hold the accepted path."""
    w = I.small_workload(890, V=3000, H=128, D=4, W=6, K=4, B=24, beta=-0.2, bf16=True)
    inp = I.make_inputs(w)
    dev = dtl.weights_to_device(inp, True)
    ctx = gu.make_ctx(w)
    g = np.random.default_rng(77)
    Hq, Hkv, dh, P, B = 8, 2, 128, 16, w.B
    cache = dtl.KVCache(2, 64, page_tokens=P, Hkv=Hkv, dh=dh)
    table, lens = torch.full((2, 20), -1, dtype=torch.int32, device="cuda"), cu([0, 0])
    bf = lambda *s: torch.from_numpy(g.standard_normal(s)).to(torch.bfloat16).cuda()  # noqa: E731
    # a prompt of 45 tokens in row 0
    assert host(cache.reserve(table, lens, cu([45, 0]))).tolist() == [1, 1]
    K0, V0 = bf(2, 45, Hkv, dh), bf(2, 45, Hkv, dh)
    for layer in range(2):
        cache.append(layer, K0, V0, table, lens, count=cu([45, 0]))
    lens.copy_(cu([45, 0]))
    q16 = lambda x: ref.values(*ref.quantise(host(x.double())))  # noqa: E731
    held = [list(q16(K0)[0]), list(q16(V0)[0])]       # what row 0 should hold
    for step in range(3):
        tree = ctx.build(dev["z"], dev["state0"], dev["A"], dev["E"], dev["Wout"], D=w.D, W=w.W, K=w.K, B=B, beta=w.beta)
        ctx.sync()
        assert host(cache.reserve(table, lens, cu([B + 1, 0])))[0] == 1
        K, V, Q = bf(1, B + 1, Hkv, dh), bf(1, B + 1, Hkv, dh), bf(1, B + 1, Hq, dh)
        for layer in range(2):
            cache.append(layer, K, V, table[:1], lens[:1])
        root = lens[:1] + 1                              # the root belongs to the prefix
        n = tree["n_out"]
        O = cache.attention(1, Q, table[:1], root, mask=tree["mask"], n_nodes=n, max_len=45 + 3 * (B + 1) + 20)
        k, v = q16(K)[0], q16(V)[0]
        Kall, Vall = np.array(held[0] + [k[0]] + list(k[1:])), np.array(held[1] + [v[0]] + list(v[1:]))
        nn = int(n[0])
        check_rows(host(O.double()), host(Q.double()), [len(held[0]) + 1], [nn],
                   host(tree["mask"]).view(np.uint32), [(Kall[:len(held[0]) + 1 + nn], Vall[:len(held[0]) + 1 + nn])], dh ** -0.5)
        # the target's logits: the drawn tokens mostly follow the tree
        t = {x: host(y)[0] for x, y in tree.items() if x != "n_out"}
        logits = g.standard_normal((B + 1, w.V)).astype(np.float32)
        for u in range(-1, nn):
            kids = np.flatnonzero(t["parent"][:nn] == u)
            if len(kids) and u < nn - 1:
                logits[u + 1, t["token"][kids[-1]]] += 30
        got = dtl.sample(torch.from_numpy(logits).cuda(), torch.rand(B + 1, device="cuda"), rows_per_req=B + 1,
                         temperature=torch.full((1,), 0.7, device="cuda"), top_p=torch.full((1,), 0.9, device="cuda"))
        acc = dtl.accept(tree["parent"], tree["token"], n, got["token"].view(1, B + 1), max_len=w.D)
        want = oracle.accept(t["parent"], t["token"], nn, host(got["token"]))
        assert int(acc["len"][0]) == want["len"] >= 1
        cache.commit(table[:1], root, acc["nodes"], acc["len"])
        lens[:1] = root
        held[0] += [k[0]] + [k[1 + i] for i in want["nodes"]]
        held[1] += [v[0]] + [v[1 + i] for i in want["nodes"]]
        cache.release(table, lens, cu([0]), lens[:1].clone())
        assert int(lens[0]) == len(held[0])
        for layer in range(2):
            rk, rv = cache.read(layer, table[:1], cu([0]), len(held[0]))
            assert np.array_equal(host(rk.double())[0], np.array(held[0]))
            assert np.array_equal(host(rv.double())[0], np.array(held[1]))
    ctx.close()
    # row 1 goes on from row 0; what row 0 then writes does not reach it
    assert host(cache.fork(table, lens, cu([0]), cu([1]))).tolist() == [1]
    cache.reserve(table, lens, cu([30, 30]))
    cache.append(0, bf(2, 30, Hkv, dh), bf(2, 30, Hkv, dh), table, lens, count=cu([30, 0]))
    rk, _ = cache.read(0, table[1:], cu([0]), len(held[0]))
    assert np.array_equal(host(rk.double())[0], np.array(held[0]))
    cache.release(table, lens, cu([0, 1]), cu([0, 0]))
    cache.check()
    assert not host(cache.refs).any()
