"""Steps of speculative decoding with a target that attends through a sliding
window and sampled drafts, every operator of a step in a row: page plans, packed
writes, window attention of draft trees, verification, commit; called one after the
other and as one captured graph."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from speculative_decoding_draft_06_gb300 import dartree as dtl
from tests import cache_ref as ref
from tests import verify_ref
from tests.test_gpu_cache import cu, host
from tests.test_gpu_verify_draft import draw_tokens, f32, tree
from tests.test_gpu_window_attention import check_request, visible

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("captured", [False, True])
@pytest.mark.parametrize("Hq, Hkv, dh, P, window, sinks", [(8, 2, 64, 16, 20, 4), (3, 3, 128, 32, 100, 0)])
def test_steps(Hq, Hkv, dh, P, window, sinks, captured):
    g = np.random.default_rng(Hq * P)
    R, B, V, width, pages, steps, prompts = 3, 12, 60, 20, 30, 12, [70, 3, 41]
    T, most = R * (B + 1) + 1, 9
    cache = dtl.KVCache(1, pages, page_tokens=P, Hkv=Hkv, dh=dh)
    table, lens = cu(np.full((R, width), -1)), cu([0] * R)
    bf16 = lambda *shape: torch.from_numpy(g.standard_normal(shape)).to(torch.bfloat16)  # noqa: E731
    # ---- the prompts
    K, Vv = bf16(sum(prompts), Hkv, dh), bf16(sum(prompts), Hkv, dh)
    out = cache.plan(table, lens, cu(prompts), max_tokens=sum(prompts), offset=0, window=window, sinks=sinks)
    assert host(out["ok"]).all()
    cache.append_slots(0, K.cuda(), Vv.cuda(), out["slot"])
    at = np.concatenate([[0], np.cumsum(prompts)])
    value = lambda x: ref.values(*ref.quantise(x.double().numpy()))  # noqa: E731
    kept = [[value(K)[at[r]:at[r + 1]], value(Vv)[at[r]:at[r + 1]]] for r in range(R)]
    lens.copy_(cu(np.array(prompts) + 1))                 # the next token, not yet in the cache, is the root
    # ---- the steps
    words = (B + 31) // 32
    s = dict(count=cu([1] * R), K=bf16(T, Hkv, dh).cuda(), V=bf16(T, Hkv, dh).cuda(), q=bf16(T, Hq, dh).cuda(),
             mask=cu(np.zeros((R, B, words))), parent=cu(np.full((R, B), -1)), token=cu(np.full((R, B), -1)),
             n=cu([0] * R), z=torch.zeros(R, B + 1, V, device="cuda"), d=torch.zeros(R, B + 1, V, device="cuda"),
             u=torch.zeros(R, B + 1, device="cuda"), T=f32([0.9, 0.0, 1.2]), p=f32([1.0, 1.0, 0.9]))

    def step():
        plan = cache.plan(table, lens, s["count"], max_tokens=T, window=window, sinks=sinks)
        cache.append_slots(0, s["K"], s["V"], plan["slot"])
        O = cache.window_attention(0, s["q"], table, lens, start=plan["start"], max_rows=B + 1, mask=s["mask"],
                                   max_len=width * P, window=window, sinks=sinks)
        got = dtl.verify(s["parent"], s["token"], s["n"], s["z"], s["d"], s["u"], max_len=most,
                         temperature=s["T"], top_p=s["p"])
        cache.commit(table, lens, got["nodes"], got["len"], extra=1)
        return plan, O, got

    graph, result, accepted = None, None, 0
    for k in range(steps):
        n = g.integers(0, B + 1, R)
        n[k % R] = B
        par, tok, anc = np.full((R, B), -1), np.full((R, B), -1), np.zeros((R, B, words * 32), bool)
        z = (g.standard_normal((R, B + 1, V)) * 2).astype(np.float32)
        d = (z + g.standard_normal(z.shape) * 0.5).astype(np.float32)
        for r in range(R):
            c = int(n[r])
            p, nth = tree(g, B, 3, most)
            par[r, :c] = p[:c]
            tok[r, :c] = draw_tokens(g, p[:c], nth[:c], d[r], 1.0)
            for i in range(c):
                if p[i] >= 0:
                    anc[r, i] = anc[r, p[i]]
                anc[r, i, i] = True
        u = g.random((R, B + 1)).astype(np.float32)
        mask = (anc.reshape(R, B, words, 32) * (1 << np.arange(32, dtype=np.int64))).sum(-1).astype(np.uint32).view(np.int32)
        count = n + 1
        new = dict(count=cu(count), K=bf16(T, Hkv, dh), V=bf16(T, Hkv, dh), q=bf16(T, Hq, dh), mask=cu(mask), parent=cu(par),
                   token=cu(tok), n=cu(n), z=torch.from_numpy(z), d=torch.from_numpy(d), u=torch.from_numpy(u))
        for name, x in new.items():
            s[name].copy_(x)
        if not captured or k == 0:
            result = step()
        else:
            if graph is None:
                torch.cuda.synchronize()
                graph = torch.cuda.CUDAGraph()
                with torch.cuda.graph(graph):
                    result = step()
            graph.replay()
        torch.cuda.synchronize()
        cache.check()
        plan, O, got = result
        assert host(plan["ok"]).all()
        O, got = host(O.double()), {name: host(x) for name, x in got.items()}
        Kv, Vv = value(new["K"]), value(new["V"])
        at = np.concatenate([[0], np.cumsum(count)])
        assert np.array_equal(host(plan["start"]), at) and not O[at[R]:].any()
        for r in range(R):
            L, c, rows = len(kept[r][0]), int(n[r]), slice(at[r], at[r + 1])
            Ks, Vs = (np.concatenate([kept[r][i], x[rows]]) for i, x in ((0, Kv), (1, Vv)))
            check_request(O[rows], new["q"][rows].double().numpy(), Ks, Vs, visible(L, c + 1, window, sinks, anc[r, :c, :c]),
                          dh ** -0.5)
            rule = dict(T=float(host(s["T"])[r]), p=float(host(s["p"])[r]))
            nodes, t, prob, tol, close = verify_ref.verify(par[r], tok[r], c, z[r], d[r], u[r], **rule)
            took = int(got["len"][r])
            if not close:
                assert (took, got["bonus"][r]) == (len(nodes), t) and abs(got["prob"][r] - prob) <= tol
                assert got["nodes"][r].tolist() == nodes + [-1] * (most - len(nodes))
            path = [0] + [1 + int(i) for i in got["nodes"][r][:took]]
            kept[r] = [np.concatenate([x, y[rows][path]]) for x, y in zip(kept[r], (Kv, Vv))]
            assert host(lens)[r] == len(kept[r][0]) + 1
            accepted += took
        t, refs = host(table), host(cache.refs)
        assert np.array_equal(np.bincount(t[t >= 0], minlength=pages), refs)
        # what a row holds: the sinks' pages, the window's, the step's (a page each begun and left)
        assert (t >= 0).sum(1).max() <= -(-sinks // P) + (window + 2 * (B + 1)) // P + 2 or k < 1
    assert accepted > 0
    cache.release(table, lens, cu([0, 1, 2]), cu([0] * R))
    cache.check()
    assert not host(cache.refs).any()


def test_plan_on_another_stream_and_in_a_graph():
    """The same results from a call on the current stream, one on another stream, a
    captured one, and one whose outputs are written again."""
    R, P, pages, width, T = 5, 16, 40, 12, 90
    g = np.random.default_rng(9)
    first, count = g.integers(0, 60, R), g.integers(0, 20, R)
    want = None
    for how in ("plain", "stream", "graph", "again"):
        cache = dtl.KVCache(1, pages, page_tokens=P, Hkv=1, dh=64)
        table, lens = cu(np.full((R, width), -1)), cu([0] * R)
        out = cache.plan(table, lens, cu(first), max_tokens=400, offset=0)
        lens.copy_(cu(first))
        n = cu(count)
        ask = dict(max_tokens=T, offset=0, window=20, sinks=3)
        torch.cuda.synchronize()
        if how == "plain":
            out = cache.plan(table, lens, n, **ask)
        elif how == "stream":
            side = torch.cuda.Stream()
            out = cache.plan(table, lens, n, stream=side, **ask)
            side.synchronize()
        elif how == "graph":
            graph = torch.cuda.CUDAGraph()
            before = host(table), host(cache.refs)
            with torch.cuda.graph(graph):
                out = cache.plan(table, lens, n, **ask)
            for _ in range(2):                             # (from the same state: the same again)
                table.copy_(cu(before[0]))
                cache.refs.copy_(cu(before[1]))
                graph.replay()
            torch.cuda.synchronize()
        else:
            out = {k: torch.full((m,), 7, dtype=torch.int32, device="cuda")
                   for k, m in (("ok", R), ("start", R + 1), ("row", T), ("pos", T), ("slot", T))}
            assert cache.plan(table, lens, n, out=out, **ask) is out
        cache.check()
        got = [host(x) for x in (*out.values(), table, cache.refs)]
        if want is None:
            want = got
        assert all(np.array_equal(a, b) for a, b in zip(got, want)), how


def test_numbers_past_32_bits():
    """Windows and sinks behind the last position are as good as it; offsets, bounds
    and row numbers that do not fit are refused, not cut off."""
    cache = dtl.KVCache(1, 8, page_tokens=16, Hkv=1, dh=64)
    table, lens, big = cu(np.arange(4)[None]), cu([50]), 1 << 32
    cache.refs[:4] = 1
    g = torch.Generator().manual_seed(1)
    cache.append(0, *(torch.randn(1, 50, 1, 64, generator=g).bfloat16().cuda() for _ in range(2)), table, cu([0]))
    q = torch.randn(1, 1, 2, 64, generator=g).bfloat16().cuda()
    attend = lambda **a: host(cache.window_attention(0, q, table, lens, **{"max_len": 50, **a}).double())  # noqa: E731
    all_ = attend()
    assert all_.any()
    for a in (dict(window=big), dict(window=big + 1), dict(window=1 << 31), dict(window=1, sinks=big), dict(window=1, sinks=1 << 31)):
        assert np.array_equal(attend(**a), all_)
    for a in (dict(offset=big), dict(offset=-big - 1), dict(max_len=big), dict(sinks=-1), dict(window=0), dict(max_len=-1)):
        with pytest.raises(ValueError):
            attend(**a)
    with pytest.raises(ValueError):
        cache.window_attention(0, q[0], table, lens, start=cu([0, 1]), max_rows=big + 1, max_len=50)
    before = host(table)
    plan = lambda **a: cache.plan(table, lens, cu([1]), **{"max_tokens": 1, **a})  # noqa: E731
    for a in (dict(window=big + 1), dict(window=1, sinks=big)):
        assert host(plan(**a)["ok"]).all() and np.array_equal(host(table), before)
    for a in (dict(offset=big), dict(max_tokens=big), dict(max_tokens=-1), dict(window=0), dict(sinks=-1)):
        with pytest.raises(ValueError):
            plan(**a)
    cache.check()


def test_fork_of_a_row_behind_its_window():
    """A row whose window has left pages behind is forked: both see the same, and
    what they held goes back."""
    Hq, Hkv, dh, P, window, sinks, L = 4, 2, 64, 16, 30, 0, 133
    g = np.random.default_rng(21)
    cache = dtl.KVCache(1, 30, page_tokens=P, Hkv=Hkv, dh=dh)
    table, lens = cu(np.full((2, 12), -1)), cu([0, 0])
    K, V = (torch.from_numpy(g.standard_normal((L, Hkv, dh))).to(torch.bfloat16) for _ in range(2))
    for a, n in ((0, 120), (120, L - 120)):
        out = cache.plan(table, lens, cu([n, 0]), max_tokens=n, offset=0, window=window, sinks=sinks)
        cache.append_slots(0, K[a:a + n].cuda(), V[a:a + n].cuda(), out["slot"])
        lens[0] += n
    assert (table[0, :5] == -1).all() and (table[0, 6:9] >= 0).all()
    assert host(cache.fork(table, lens, cu([0]), cu([1]))).tolist() == [1]
    q = torch.from_numpy(g.standard_normal((1, 1, Hq, dh))).to(torch.bfloat16)
    O = host(cache.window_attention(0, q.expand(2, -1, -1, -1).contiguous().cuda(), table, lens, max_len=L, window=window).double())
    k, v = (ref.values(*ref.quantise(x.double().numpy())) for x in (K, V))
    for r in range(2):
        check_request(O[r], q[0].double().numpy(), k, v, visible(L - 1, 1, window, sinks), dh ** -0.5)
    cache.release(table, lens, cu([0, 1]), cu([0, 0]))
    cache.check()
    assert not host(cache.refs).any() and (host(table) == -1).all()


def test_far_pages_and_rows():
    """Pages and query rows that lie more than 2^32 bytes apart."""
    Hq, Hkv, dh, P, pages, window, L, n = 8, 8, 128, 128, 30000, 200, 300, 40
    g = np.random.default_rng(22)
    cache = dtl.KVCache(1, pages, page_tokens=P, Hkv=Hkv, dh=dh)
    assert pages * cache.page_bytes > 1 << 32
    cache.refs[:pages - 4] = 1
    table, lens = cu(np.full((1, 5), -1)), cu([0])
    K, V = (torch.from_numpy(g.standard_normal((L, Hkv, dh))).to(torch.bfloat16) for _ in range(2))
    out = cache.plan(table, lens, cu([L]), max_tokens=L, offset=0)
    assert host(table).tolist() == [[pages - 4, pages - 3, pages - 2, -1, -1]]
    cache.append_slots(0, K.cuda(), V.cuda(), out["slot"])
    step = 1 << 26                                          # elements between rows: 40 of them pass 2^32 bytes
    q = torch.from_numpy(g.standard_normal((n, Hq, dh))).to(torch.bfloat16)
    far = torch.empty(n * step, dtype=torch.bfloat16, device="cuda").as_strided((n, Hq, dh), (step, dh, 1))
    far.copy_(q)
    k, v = (ref.values(*ref.quantise(x.double().numpy())) for x in (K, V))
    for rows in (n, 3):                                     # the tensor cores' kernel, the few rows'
        O = host(cache.window_attention(0, far[n - rows:], table, cu([L - rows]), start=cu([0, rows]), max_rows=rows, max_len=L,
                                        window=window, offset=0).double())
        check_request(O, q[n - rows:].double().numpy(), k, v, visible(L - rows, rows, window, 0), dh ** -0.5)
    cache.check()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_far_logits(dtype):
    """Requests' and nodes' logits that lie more than 2^32 bytes apart."""
    g = np.random.default_rng(23)
    R, B, V, row, req = 2, 3, 700, 1 << 29, (1 << 31) + (1 << 20)
    z = torch.from_numpy(g.standard_normal((R, B + 1, V)) * 2).to(dtype)
    d = torch.from_numpy(z.float().numpy() + g.standard_normal(z.shape) * 0.2).to(dtype)
    far = torch.empty(req + B * row + V, dtype=dtype, device="cuda").as_strided((R, B + 1, V), (req, row, 1))
    near = torch.empty(R, B + 1, V, dtype=dtype, device="cuda")
    u = f32(g.random((R, B + 1)) * 0.2)
    tok = cu([draw_tokens(g, np.arange(B) - 1, np.zeros(B, int), d[r].float().numpy(), 1.0) for r in range(R)])
    got = []
    for logits, draft in ((far, near), (near, far)):
        logits.copy_(z)
        draft.copy_(d)
        got.append(dtl.verify(None, tok, cu([B] * R), logits, draft, u, max_len=B, top_p=f32([0.99] * R)))
    want = dtl.verify(None, tok, cu([B] * R), z.cuda(), d.cuda(), u, max_len=B, top_p=f32([0.99] * R))
    assert host(want["len"]).sum() > 0
    for x in got:
        assert all(np.array_equal(host(x[k]), host(want[k])) for k in want)
