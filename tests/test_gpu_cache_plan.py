"""Page tables and slot maps from request lengths, packed writes, and a few
steps of a served target with a sliding window, against references that take
one row, page and token at a time."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from speculative_decoding_draft_06_gb300 import dartree as dtl
from tests import cache_ref as ref
from tests.test_gpu_cache import cu, hard_values, host, tables
from tests.test_gpu_window_attention import check_request, visible

pytestmark = pytest.mark.gpu


def plan_ref(table, refs, lens, count, P, offset, window, sinks, T):
    """The definition, in place on table and refs -> ok, start, row, pos, slot."""
    R, width = table.shape
    pages = len(refs)
    valid, tokens, full = [], [], 0
    for r in range(R):
        f, n = int(lens[r]) + offset, int(count[r])
        good = lens[r] >= 0 and n >= 0 and f >= 0 and f + n <= 2 ** 31 - 1
        if good and n > 0:
            full += n
            good = full <= T
        valid.append(good)
        tokens.append(n if good else 0)
    if window:
        for r in range(R):
            if not valid[r]:
                continue
            for j in range(width):
                if j * P >= sinks and j * P + P - 1 <= int(lens[r]) + offset - window and table[r, j] != -1:
                    if 0 <= table[r, j] < pages and refs[table[r, j]] > 0:
                        refs[table[r, j]] -= 1
                    table[r, j] = -1
    held, lacks = refs.copy(), []
    for r in range(R):
        f, n = int(lens[r]) + offset, tokens[r]
        need = list(range(f // P, -(-(f + n) // P))) if valid[r] and n else []
        bad = not valid[r] or any(j >= width for j in need)
        got = [] if bad else [table[r, j] for j in need]
        k = 0
        while k < len(got) and got[k] >= 0:
            k += 1
        bad = bad or any(x >= 0 for x in got[k:]) or any(x >= pages or held[x] > 1 for x in got[:k])
        lacks.append(None if bad else need[k:])
    ok, free, out = np.zeros(R, np.int32), int((refs == 0).sum()), False
    for r in range(R):
        if lacks[r] is None:
            continue
        out = out or len(lacks[r]) > free
        if lacks[r] and out:
            continue
        ok[r] = 1
        for j in lacks[r]:
            page = int(np.flatnonzero(refs == 0)[0])
            table[r, j], refs[page] = page, 1
            free -= 1
    start = np.concatenate([[0], np.cumsum(tokens)])
    row, pos, slot = (np.full(T, -1) for _ in range(3))
    for r in range(R):
        for i in range(tokens[r]):
            t, at = start[r] + i, int(lens[r]) + offset + i
            row[t], pos[t] = r, at
            if ok[r]:
                slot[t] = table[r, at // P] * P + at % P
    return ok, start, row, pos, slot


CASES = [  # R, width, pages, P, offset, window, sinks, most tokens, T
    (1, 3, 4, 16, 0, None, 0, 20, 20), (1, 9, 12, 16, -1, 30, 4, 40, 50), (5, 8, 30, 32, -1, 1, 0, 60, 200),
    (17, 12, 90, 16, 0, 50, 17, 40, 300), (64, 7, 200, 64, -1, 70, 64, 100, 3000), (33, 6, 40, 128, 3, None, 0, 300, 9000),
    (300, 10, 1500, 16, -1, 40, 4, 9, 1000), (9, 30, 9000, 16, 0, 100, 1, 60, 40000), (700, 20, 12000, 16, -1, 33, 0, 30, 33000),
    (4096, 4, 40000, 16, 0, 16, 0, 20, 50000), (3, 700, 1500, 16, 0, 64, 100, 200, 600), (2, 5, 10, 16, 0, 1 << 30, 0, 30, 60),
    (40, 5, 100, 32, -1, 20, 1 << 30, 10, 0),
]


@pytest.mark.parametrize("case", range(len(CASES)))
def test_plan(case):
    R, width, pages, P, offset, window, sinks, most, T = CASES[case]
    g = np.random.default_rng(7000 + case)
    have = g.integers(0, width + 1, R)
    have = np.where(np.cumsum(have) <= pages * 3 // 4, have, 0)
    table, refs = tables(g, have, pages, width)
    lens = np.array([g.integers(max(0, h * P - P), h * P + 1) for h in have])
    count = g.integers(0, most + 1, R)
    # odd rows: negative lengths and counts, pages shared with a later row, holes, bad numbers, counted tokens that have no page
    for r in range(R):
        kind = g.integers(0, 14)
        if kind == 0:
            lens[r] = -1
        elif kind == 1:
            count[r] = -3
        elif kind == 2 and have[r] > 1:
            lens[r] = int(g.integers(0, have[r] * P))          # cut back
        elif kind == 3 and r + 1 < R and have[r]:
            shared = table[r].copy()
            back = table[r + 1][table[r + 1] >= 0]
            refs[back] -= 1
            table[r + 1] = shared
            refs[shared[shared >= 0]] += 1
            lens[r + 1] = lens[r]
        elif kind == 4 and have[r] > 2:
            refs[table[r, have[r] - 2]] -= 1
            table[r, have[r] - 2] = -1
            lens[r] = (have[r] - 3) * P + 1
        elif kind == 5 and have[r]:
            refs[table[r, have[r] - 1]] -= 1
            table[r, have[r] - 1] = pages + 7
    cache = dtl.KVCache(1, pages, page_tokens=P, Hkv=1, dh=64, refs=cu(refs))
    t, ln = cu(table), cu(lens)
    want_table, want_refs = table.copy(), refs.copy()
    want = plan_ref(want_table, want_refs, lens, count, P, offset, window, sinks, T)
    out = cache.plan(t, ln, cu(count), max_tokens=T, offset=offset, window=window, sinks=sinks)
    torch.cuda.synchronize()
    for name, w in zip(("ok", "start", "row", "pos", "slot"), want):
        assert np.array_equal(host(out[name]), w), name
    assert np.array_equal(host(t), want_table)
    assert np.array_equal(host(cache.refs), want_refs)
    assert np.array_equal(host(ln), lens)
    cache.err.zero_()
    # once more: the same maps, nothing taken (rows that were refused for pages may fare better or not, so only then)
    if (want[0] == 1).all():
        reused = {k: torch.full_like(v, 99) for k, v in out.items()}
        again = cache.plan(t, ln, cu(count), max_tokens=T, offset=offset, window=window, sinks=sinks, out=reused)
        assert again is reused
        assert all(np.array_equal(host(again[k]), host(out[k])) for k in out)
        assert np.array_equal(host(t), want_table) and np.array_equal(host(cache.refs), want_refs)


def test_plan_runs_out_of_pages():
    """The row the pages run out in gives back what it got; rows that need none
    are served."""
    P, width, pages = 16, 10, 9
    table = np.full((4, width), -1, np.int32)
    refs = np.zeros(pages, np.int32)
    table[3, :2] = [4, 7]
    refs[[4, 7]] = 1
    lens, count = np.array([0, 0, 0, 20]), np.array([40, 100, 10, 5])
    cache = dtl.KVCache(1, pages, page_tokens=P, Hkv=1, dh=64, refs=cu(refs))
    t, ln = cu(table), cu(lens)
    out = cache.plan(t, ln, cu(count), max_tokens=155, offset=0)
    assert host(out["ok"]).tolist() == [1, 0, 0, 1]
    assert host(t)[0, :4].tolist() == [0, 1, 2, -1] and (host(t)[1:3] == -1).all()
    assert host(cache.refs).tolist() == [1, 1, 1, 0, 1, 0, 0, 1, 0]
    assert (host(out["slot"])[40:150] == -1).all() and host(out["pos"])[40:44].tolist() == [0, 1, 2, 3]
    assert host(out["slot"])[150:].tolist() == [7 * 16 + 4 + i for i in range(5)]


PUTS = [(1, 1, 128, 16, 0, 0), (37, 3, 64, 32, 2, -4), (500, 8, 128, 64, 0, 0), (1023, 2, 64, 128, -3, 5)]


@pytest.mark.parametrize("T, Hkv, dh, P, ke, ve", PUTS)
def test_append_slots(T, Hkv, dh, P, ke, ve):
    """Scattered slots, some of them none, one outside the pool, one page that is
    held twice; K and V sliced from a fused projection."""
    g = np.random.default_rng(T)
    pages = T // P + 6
    refs = np.ones(pages, np.int32)
    refs[1] = 2
    cache = dtl.KVCache(2, pages, page_tokens=P, Hkv=Hkv, dh=dh, k_scale=2.0 ** ke, v_scale=2.0 ** ve, refs=cu(refs))
    slot = g.permutation(pages * P)[:T]
    slot[slot // P == 1] = -5
    if T > 10:
        slot[3], slot[5] = -1, pages * P + 2
        slot[7] = P + 3
    fused = hard_values(g, (T, (2 * Hkv + 1) * dh)).cuda()
    K, V = fused[:, :Hkv * dh].view(T, Hkv, dh), fused[:, Hkv * dh:2 * Hkv * dh].view(T, Hkv, dh)
    cache.append_slots(1, K, V, cu(slot))
    if T > 10:
        with pytest.raises(dtl.DartreeError):
            cache.check()
    cache.check()
    pool = host(cache.pool)
    assert not pool[0].any() and not pool[1, 1].any()
    k, v = ([ref.quantise(x.double().cpu().numpy()[i], 2.0 ** e) for i in range(T)] for x, e in ((K, ke), (V, ve)))
    written = np.zeros((pages, P), bool)
    for i, s in enumerate(slot):
        if s < 0 or s >= pages * P or s // P == 1:
            continue
        written[s // P, s % P] = True
        views = ref.page_views(pool[1, s // P], P, Hkv, dh)
        for at, want in zip(views, (k[i][0], k[i][1], v[i][0], v[i][1])):
            x = at[:, s % P]
            # (a zero's sign does not matter)
            assert np.array_equal(np.where(x == 8, 0, x), np.where(want == 8, 0, want)), (i, s)
    for page in range(pages):
        for at in ref.page_views(pool[1, page], P, Hkv, dh):
            assert not at[:, ~written[page]].any()


def test_refusals():
    cache = dtl.KVCache(1, 8, page_tokens=16, Hkv=2, dh=64)
    t, ln, n = cu(np.full((2, 4), -1)), cu([3, 4]), cu([1, 1])
    for k in (dict(max_tokens=-1), dict(max_tokens=4, window=0), dict(max_tokens=4, sinks=-1)):
        with pytest.raises((ValueError, dtl.DartreeError)):
            cache.plan(t, ln, n, **k)
    with pytest.raises(ValueError):
        cache.plan(t, ln, cu([1]), max_tokens=4)
    with pytest.raises(ValueError):
        cache.plan(t, ln, n, max_tokens=4, out=cache.plan(t, ln, cu([0, 0]), max_tokens=5))
    x = torch.zeros(5, 2, 64, dtype=torch.bfloat16, device="cuda")
    s = cu([0, 1, 2, 3, 4])
    for K, V, sl in ((x.float(), x, s), (x, x.cpu(), s), (x[:, :1], x[:, :1], s), (x, x[:4], s), (x, x, s[:4]), (x, x, s.long()),
                     (x, x.transpose(0, 1).contiguous().transpose(0, 1), s)):
        with pytest.raises((TypeError, ValueError)):
            cache.append_slots(0, K, V, sl)
    with pytest.raises(dtl.DartreeError):
        cache.append_slots(1, x, x, s)
    assert not host(cache.refs).any() and (host(t) == -1).all()


@pytest.mark.parametrize("window, sinks, P", [(40, 4, 16), (100, 0, 32), (None, 0, 64)])
def test_steps_of_a_served_target(window, sinks, P):
    """Prompts in pieces, then drafted chains of which a part is kept, then
    single tokens, all packed: plan, append_slots, window_attention, release;
    the attention is the formula's over everything that was ever kept, and the
    windows' pages go back."""
    g = np.random.default_rng(P)
    R, Hq, Hkv, dh, width, pages = 3, 4, 2, 64, 40, 60
    cache = dtl.KVCache(1, pages, page_tokens=P, Hkv=Hkv, dh=dh)
    table, lens = cu(np.full((R, width), -1)), cu([0] * R)
    kept = [[np.zeros((0, Hkv, dh)), np.zeros((0, Hkv, dh))] for _ in range(R)]
    most = 70
    steps = [[70, 33, 5], [64, 1, 70], [1, 70, 2], [9, 9, 1], [4, 1, 9], [0, 1, 1], [1, 1, 1], [9, 5, 9], [70, 0, 1]]
    for n in steps:
        out = cache.plan(table, lens, cu(n), max_tokens=sum(n) + 2, offset=0, window=window, sinks=sinks)
        assert host(out["ok"]).all()
        T = sum(n) + 2
        K, V = (torch.from_numpy(g.standard_normal((T, Hkv, dh))).to(torch.bfloat16) for _ in range(2))
        q = torch.from_numpy(g.standard_normal((T, Hq, dh))).to(torch.bfloat16)
        cache.append_slots(0, K.cuda(), V.cuda(), out["slot"])
        top = max(len(k[0]) + c for k, c in zip(kept, n))
        O = host(cache.window_attention(0, q.cuda(), table, lens, start=out["start"], max_rows=most, max_len=top,
                                        window=window, sinks=sinks, offset=0).double())
        cache.check()
        k, v = (ref.values(*ref.quantise(x.double().numpy())) for x in (K, V))
        at, keep = 0, []
        for r, c in enumerate(n):
            L = len(kept[r][0])
            Ks, Vs = (np.concatenate([kept[r][i], x[at:at + c]]) for i, x in ((0, k), (1, v)))
            if c:
                check_request(O[at:at + c], q[at:at + c].double().numpy(), Ks, Vs, visible(L, c, window, sinks), dh ** -0.5)
            m = int(g.integers(1, c + 1)) if 1 < c < 10 else c            # a drafted chain is kept in part
            kept[r] = [Ks[:L + m], Vs[:L + m]]
            keep.append(L + m)
            at += c
        assert not O[at:].any()
        lens.copy_(cu(keep))
        cache.release(table, lens, cu([0, 1, 2]), lens.clone())
        cache.check()
        t, refs = host(table), host(cache.refs)
        assert np.array_equal(np.bincount(t[t >= 0], minlength=pages), refs)
        for r in range(R):
            f = keep[r] - n[r] if n[r] == 0 else keep[r]
            assert (t[r, -(-keep[r] // P):] == -1).all()
            if window:
                # what the step's plan let go: pages behind the window of its first token
                assert (t[r] >= 0).sum() <= -(-sinks // P) + (window + most) // P + 3, f
    if window:
        assert host(cache.refs).sum() < sum(-(-x // P) for x in keep)
