"""The paged 4-bit cache on the GPU: writing, reading and the page operations
against the references in 64 bits (tests/cache_ref.py)."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from speculative_decoding_draft_06_gb300 import dartree as dtl
from tests import cache_ref as ref

pytestmark = pytest.mark.gpu

BAD = 16


def cu(a):
    return torch.from_numpy(np.ascontiguousarray(a, np.int32)).cuda()


def host(t):
    return t.cpu().numpy()


def tables(g, held, pages, width):
    ids, table, at = g.permutation(pages), np.full((len(held), width), -1, np.int32), 0
    for r, k in enumerate(held):
        table[r, :k] = ids[at:at + k]
        at += k
    refs = np.zeros(pages, np.int32)
    refs[table[table >= 0]] = 1
    return table, refs


def hard_values(g, shape):
    """bf16 data with what is hard for the format: ties of codes and scales,
    huge and tiny blocks, zeros, infinities and NaN."""
    x = g.standard_normal(shape) * 10.0 ** g.integers(-3, 3, (*shape[:-1], 1))
    b = x.reshape(-1, 16)
    kind = g.integers(0, 12, len(b))
    b[kind == 0] = 0.0
    for i in np.flatnonzero(kind == 1):   # exact ties: codes' midpoints times a scale, and 6 scales
        s = ref.E4M3[g.integers(1, 127)]
        b[i] = g.choice([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, -0.25, -5.0, 1.0, 6.0], 16) * s
        b[i, 0] = 6 * s
    for i in np.flatnonzero(kind == 2):   # max / 6 half-way between two scales
        j = g.integers(0, 126)
        b[i] = g.uniform(-1, 1, 16)
        b[i, 3] = 6 * (ref.E4M3[j] + ref.E4M3[j + 1]) / 2
    b[kind == 3] *= 1e6
    b[kind == 4] *= 1e-6
    b[kind == 5, 2] = np.nan
    b[kind == 6, 5] = np.inf
    b[kind == 6, 6] = -np.inf
    return torch.from_numpy(x).to(torch.bfloat16)


WRITES = [  # R, n, Hkv, dh, P, unit exponents
    (1, 1, 1, 128, 16, 0, 0), (3, 7, 2, 64, 16, 0, 0), (2, 65, 3, 128, 64, 3, -5), (2, 130, 8, 64, 128, 0, -20),
    (5, 33, 1, 128, 32, 10, 1),
]


@pytest.mark.parametrize("case", range(len(WRITES)))
def test_append_and_read(case):
    """Codes, scales and values are exactly the reference's."""
    R, n, Hkv, dh, P, ke, ve = WRITES[case]
    g = np.random.default_rng(case)
    lens = g.integers(0, 3 * P, R)
    lens[0] = 0
    held = -(-(lens + n) // P)
    table, refs = tables(g, held, int(held.sum()) + 3, int(held.max()) + 1)
    cache = dtl.KVCache(2, len(refs), page_tokens=P, Hkv=Hkv, dh=dh, k_scale=2.0 ** ke, v_scale=2.0 ** ve, refs=cu(refs))
    cache.pool.fill_(0xA5)
    K, V = hard_values(g, (R, n, Hkv, dh)), hard_values(g, (R, n, Hkv, dh))
    cache.append(1, K.cuda(), V.cuda(), cu(table), cu(lens))
    pool = host(cache.pool)
    assert (pool[0] == 0xA5).all()                      # another layer's
    untouched = np.ones(pool.shape[1:], bool)
    got = cache.read(1, cu(table), cu(lens), n)
    cache.check()
    for x, unit, which in ((K, 2.0 ** ke, 0), (V, 2.0 ** ve, 2)):
        x64 = x.double().numpy()
        code, sc = ref.quantise(x64, unit)
        val = host(got[which // 2].double())
        assert np.array_equal(val, ref.values(code, sc, unit))
        for r in range(R):
            for i in range(n):
                pos = int(lens[r]) + i
                page = table[r, pos // P]
                v = ref.page_views(pool[1, page], P, Hkv, dh)
                same = (v[which][:, pos % P] & 7) == (code[r, i] & 7)
                sign = (v[which][:, pos % P] == code[r, i]) | np.isnan(x64[r, i])
                assert same.all() and sign.all() and np.array_equal(v[which + 1][:, pos % P], sc[r, i])
                m = np.zeros((Hkv, P, dh), np.uint8)
                m[:, pos % P] = 1
                c = untouched[page].reshape(Hkv, -1)
                at = 0
                for unit_b in (dh // 2, dh // 16) * 2:
                    c[:, at + (pos % P) * unit_b: at + (pos % P + 1) * unit_b] = False
                    at += P * unit_b
    assert (pool[1][untouched] == 0xA5).all()           # nothing beside the tokens


def test_append_slices_counts_and_skipped_rows():
    """Slices of a fused projection, an offset, counts, rows with negative
    lengths, tokens without a page."""
    g = np.random.default_rng(11)
    R, n, Hkv, dh, P = 4, 20, 2, 128, 16
    lens = np.array([30, 5, -1, 40])
    table, refs = tables(g, [4, 2, 3, 3], 20, 5)
    cache = dtl.KVCache(1, 20, page_tokens=P, Hkv=Hkv, dh=dh, refs=cu(refs))
    x = torch.randn(R, n, 4 * Hkv * dh, dtype=torch.float64).to(torch.bfloat16).cuda()
    K = x[:, :, Hkv * dh:2 * Hkv * dh].view(R, n, Hkv, dh)
    V = x[:, :, 3 * Hkv * dh:].view(R, n, Hkv, dh)
    count = np.array([20, 0, 20, 9])
    out = tuple(torch.full((R, n, Hkv, dh), 7.0, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    cache.append(0, K, V, cu(table), cu(lens), offset=-1, count=cu(count))
    cache.check()                                       # row 3: positions 39 .. 47 are mapped
    cache.read(0, cu(table), cu(lens), n, offset=-1, count=cu(count), out=out)
    cache.check()
    for got, x in zip(out, (K, V)):
        want = ref.values(*ref.quantise(host(x.double())))
        got = host(got.double())
        for r in range(R):
            c = count[r] if lens[r] >= 0 else 0
            assert np.array_equal(got[r, :c], want[r, :c]) and (got[r, c:] == 7.0).all()
    before = cache.pool.clone()
    cache.append(0, K, V, cu(table), cu(np.array([-1, 60, -5, -3])))    # row 1: no pages there
    assert torch.equal(before, cache.pool)
    with pytest.raises(dtl.DartreeError):
        cache.check()
    cache.check()
    k, v = cache.read(0, cu(table), cu(np.array([-1, 30, -5, -3])), 4, out=tuple(o[:, :4].contiguous() for o in out))
    assert (host(k.float())[1] == 0).all()              # 30, 31: never written (count 0) | 32, 33: no page
    with pytest.raises(dtl.DartreeError):
        cache.check()
    bad = table.copy()
    bad[0, 1] = 20                                      # a page that does not exist
    cache.append(0, K, V, cu(bad), cu(np.array([16, -1, -1, -1])), count=cu([16, 0, 0, 0]))
    assert torch.equal(before, cache.pool)
    with pytest.raises(dtl.DartreeError):
        cache.check()


def test_offsets_past_32_bits():
    """Pages behind the pool's first 4 GB."""
    Hkv, dh, P = 8, 128, 128
    cache = dtl.KVCache(2, 20000, page_tokens=P, Hkv=Hkv, dh=dh)       # 5.9 GB
    table = cu([[19999, 3], [14600, 19998]])
    lens = cu([100, 100])
    K = torch.randn(2, 60, Hkv, dh, device="cuda").to(torch.bfloat16)
    cache.append(1, K, -K, table, lens)
    k, v = cache.read(1, table, lens, 60)
    cache.check()
    want = ref.values(*ref.quantise(host(K.double())))
    assert np.array_equal(host(k.double()), want) and np.array_equal(host(v.double()), -want)
    cache.copy_pages(cu([19999, 3]), cu([15000, 15001]))
    k2, _ = cache.read(1, cu([[15000, 15001], [14600, 19998]]), lens, 60)
    assert torch.equal(k, k2)


def sequences(g, R, P, Hkv, dh, layers, width, pages, spare_rows=0):
    """A pool of random bytes and sequences that hold pages for their lengths
    and some more."""
    lens = np.concatenate([g.integers(0, (width - 1) * P, R), np.zeros(spare_rows, np.int64)]).astype(np.int32)
    held = -(-lens // P)
    held[:R] = np.minimum(held[:R] + g.integers(0, 2, R), width)
    table, refs = tables(g, held, pages, width)
    pool = g.integers(0, 256, (layers, pages, Hkv * P * dh // 8 * 9), dtype=np.uint8)
    cache = dtl.KVCache(layers, pages, page_tokens=P, Hkv=Hkv, dh=dh, pool=torch.from_numpy(pool).cuda(), refs=cu(refs))
    return cache, ref.Pages(pool, refs, table, lens, P), cu(table), cu(lens)


def same(cache, want, table, lens):
    assert np.array_equal(host(table), want.table)
    assert np.array_equal(host(lens), want.lens)
    assert np.array_equal(host(cache.refs), want.refs)
    assert np.array_equal(host(cache.pool), want.pool)


@pytest.mark.parametrize("seed", range(6))
def test_reserve(seed):
    """Enough pages, too few (the rows are served in order), wants that do
    not fit a row, negative lengths and wants, nothing wanted."""
    g = np.random.default_rng(seed)
    R, P, width = int(g.integers(1, 40)), int(g.choice([16, 32, 64, 128])), int(g.integers(1, 70))
    room = R * width
    cache, want, table, lens = sequences(g, R, P, 1, 64, 1, width, room + int(g.integers(0, 5000)))
    w = g.integers(0, 3 * P, R)
    w[g.random(R) < 0.2] = 0
    if seed % 2:                          # few pages: others are held
        busy = g.permutation(np.flatnonzero(want.refs == 0))
        want.refs[busy[int(g.integers(0, 6)):]] = 1
        cache.refs.copy_(cu(want.refs))
        w[g.random(R) < 0.1] = -1
        want.lens[g.random(R) < 0.1] = -1
        lens.copy_(cu(want.lens))
        w[g.random(R) < 0.1] = 2 ** 31 - 1
    ok = cache.reserve(table, lens, cu(w))
    assert np.array_equal(host(ok), want.reserve(w))
    same(cache, want, table, lens)


@pytest.mark.parametrize("seed", range(6))
def test_fork(seed):
    """Shared and copied pages, too few pages, rows that are refused."""
    g = np.random.default_rng(100 + seed)
    P, dh, Hkv = int(g.choice([16, 32, 64, 128])), int(g.choice([64, 128])), int(g.integers(1, 4))
    R, S, width = 6, 12, 5
    cache, want, table, lens = sequences(g, R, P, Hkv, dh, 3, width, 60, S)
    if seed == 0:
        want.lens[:R] = [0, P, 2 * P, 1, P - 1, P + 1]
        held = -(-want.lens[:R] // P)
        want.table[:], want.refs[:] = -1, 0
        for r in range(R):
            want.table[r, :held[r]] = 7 * r + np.arange(held[r])
            want.refs[want.table[r, :held[r]]] = 1
        table.copy_(cu(want.table)), lens.copy_(cu(want.lens)), cache.refs.copy_(cu(want.refs))
    src = g.integers(0, R, S)
    dst = R + g.permutation(S)
    if seed >= 3:                         # refusals: out of range, not empty, twice, a source
        src[0], dst[1], dst[2], dst[3], src[4] = -1, R + S, 0, dst[5], R + S
        src[6] = dst[7]
    if seed >= 4:
        busy = g.permutation(np.flatnonzero(want.refs == 0))
        want.refs[busy[2:]] = 1
        cache.refs.copy_(cu(want.refs))
    ok = cache.fork(table, lens, cu(src), cu(dst))
    assert np.array_equal(host(ok), want.fork(list(src), list(dst)))
    same(cache, want, table, lens)


@pytest.mark.parametrize("seed", range(4))
def test_release(seed):
    """After forks: shared pages stay while somebody holds them; a row listed
    twice lets each page go once."""
    g = np.random.default_rng(200 + seed)
    P = int(g.choice([16, 64]))
    cache, want, table, lens = sequences(g, 6, P, 1, 64, 1, 6, 60, 6)
    src, dst = list(range(6)), list(range(6, 12))
    cache.fork(table, lens, cu(src), cu(dst))
    want.fork(src, dst)
    rows = g.integers(-1, 13, 10)
    rows[3] = rows[4]
    keep = g.integers(0, 4 * P, 10)
    keep[::3] = 0
    keep[5] = -1 if seed == 3 else keep[5]
    cache.release(table, lens, cu(rows), cu(keep))
    want.release(rows, keep)
    same(cache, want, table, lens)
    bad = bool(((rows < 0) | (rows >= 12) | (keep < 0)).any())
    assert int(cache.err.item()) == (BAD if bad else 0)
    # everything goes: no page is held
    cache.release(table, lens, cu(list(range(12))), cu([0] * 12))
    assert not host(cache.refs).any() and (host(table) == -1).all() and not host(lens).any()


COMMITS = [(64, 128, 8, 4, 7), (16, 64, 3, 2, 16), (128, 128, 1, 1, 1), (32, 64, 2, 3, 40), (16, 128, 8, 1, 130),
           (64, 128, 2, 20, 9), (16, 64, 3, 9, 33), (32, 128, 8, 17, 60)]


@pytest.mark.parametrize("case", range(len(COMMITS)))
def test_commit(case):
    """Paths of rising ranks, from none to longer than one chunk; identity
    paths; bad ranks and rows that are left as they were."""
    P, dh, Hkv, layers, most = COMMITS[case]
    g = np.random.default_rng(300 + case)
    R, nodes_n = 7, max(150, 2 * most)
    width = -(-(40 + nodes_n) // P) + 1
    pages = R * width
    lens = g.integers(0, 40, R).astype(np.int32)
    table, refs = tables(g, -(-(lens + nodes_n) // P), pages, width)
    pool = g.integers(0, 256, (layers, pages, Hkv * P * dh // 8 * 9), dtype=np.uint8)
    cache = dtl.KVCache(layers, pages, page_tokens=P, Hkv=Hkv, dh=dh, pool=torch.from_numpy(pool).cuda(), refs=cu(refs))
    nodes = np.full((R, most), -1)
    length = g.integers(0, most + 1, R)
    length[0], length[1] = most, 0
    for r in range(R):
        nodes[r, :length[r]] = np.sort(g.choice(nodes_n, length[r], replace=False))
    nodes[2, :length[2]] = np.arange(length[2])         # already in place
    flagged = False
    if most > 3:
        length[3:7] = most
        nodes[3] = np.sort(g.choice(nodes_n, most, replace=False))
        nodes[3, 1] = nodes[3, 0]                       # not rising
        nodes[4] = np.arange(most) - 1                  # negative
        nodes[5] = np.arange(most)
        nodes[5, -1] = width * P                        # no page
        nodes[6] = np.arange(most) + 1
        lens[6] = -1
        flagged = True
    t, ln = cu(table), cu(lens)
    want = ref.Pages(pool, refs, table, lens, P)
    cache.commit(t, ln, cu(nodes), cu(length), extra=1)
    want.commit(nodes, length, 1, Hkv, dh)
    same(cache, want, t, ln)
    assert int(cache.err.item()) == (BAD if flagged else 0)


def test_a_row_cut_within_a_shared_page_does_not_grow():
    """Its next token would go into a page that the other row reads: reserve
    refuses it until the row is forked or the page is its own."""
    c = dtl.KVCache(2, 12, page_tokens=16, Hkv=1, dh=64)
    table, lens = cu(np.full((3, 6), -1)), cu([0, 0, 0])
    assert host(c.reserve(table, lens, cu([40, 0, 0]))).tolist() == [1, 1, 1]
    lens[0] = 40
    assert host(c.fork(table, lens, cu([0]), cu([1]))).tolist() == [1]
    c.release(table, lens, cu([1]), cu([20]))
    before = host(table)
    assert host(c.reserve(table, lens, cu([1, 1, 0]))).tolist() == [1, 0, 1]
    assert host(c.reserve(table, lens, cu([1, 0, 0]))).tolist() == [1, 1, 1]
    assert (host(table) == before).all()
    assert host(c.fork(table, lens, cu([1]), cu([2]))).tolist() == [1]
    assert host(c.reserve(table, lens, cu([0, 1, 30]))).tolist() == [1, 0, 1]
    t = host(table)
    assert t[2, 0] == t[0, 0] and t[2, 1] not in (t[0, 1], -1) and (t[2, 2:4] >= 0).all()
    c.release(table, lens, cu([0]), cu([0]))
    assert host(c.reserve(table, lens, cu([0, 1, 0]))).tolist() == [1, 1, 1]
    c.check()


def test_copy_pages():
    g = np.random.default_rng(7)
    Hkv, dh, P, layers, pages = 3, 64, 32, 2, 40
    pool = g.integers(0, 256, (layers, pages, Hkv * P * dh // 8 * 9), dtype=np.uint8)
    cache = dtl.KVCache(layers, pages, page_tokens=P, Hkv=Hkv, dh=dh, pool=torch.from_numpy(pool).cuda())
    src, dst = [0, 1, 1, 2, 3, -1, 5, 6], [10, 11, 12, 11, 40, 13, 14, 6]
    cache.copy_pages(cu(src), cu(dst))                  # 11 twice, 40 and -1 outside, 6 onto itself
    want = pool.copy()
    for s, d in ((0, 10), (1, 11), (1, 12), (5, 14)):
        want[:, d] = pool[:, s]
    assert np.array_equal(host(cache.pool), want)
    assert int(cache.err.item()) == BAD


def test_binding_refuses_bad_tensors():
    cache = dtl.KVCache(1, 8, page_tokens=16, Hkv=2, dh=64)
    table, lens = cu([[0, 1]]), cu([3])
    K = torch.zeros(1, 4, 2, 64, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(TypeError):
        cache.append(0, K.float(), K, table, lens)
    with pytest.raises(ValueError):
        cache.append(0, K[..., :32], K[..., :32], table, lens)
    with pytest.raises(ValueError):
        cache.append(0, K.transpose(1, 2).contiguous().transpose(1, 2), K, table, lens)
    with pytest.raises(TypeError):
        cache.append(0, K, K, table.long(), lens)
    with pytest.raises(TypeError):
        cache.read(0, table, lens.cpu(), 4)
    with pytest.raises(ValueError):
        cache.read(0, table, lens.repeat(2), 4)
    with pytest.raises(dtl.DartreeError):
        cache.append(1, K, K, table, lens)
    with pytest.raises(ValueError):
        cache.attention(0, torch.zeros(1, 3, 4, 64, dtype=torch.bfloat16, device="cuda"), table, lens, max_len=8)
    with pytest.raises(ValueError):
        dtl.KVCache(1, 8, page_tokens=16, Hkv=2, dh=64, k_scale=1.5)
    with pytest.raises(ValueError):
        dtl.KVCache(1, 8, page_tokens=20, Hkv=2, dh=64)
