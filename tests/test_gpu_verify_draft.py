"""Verification of drafted tokens on the GPU against the definition in 64 bits,
request by request."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from speculative_decoding_draft_06_gb300 import dartree as dtl
from tests import verify_ref as ref
from tests.test_gpu_cache import cu, host

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


def f32(x):
    return torch.tensor(np.asarray(x), dtype=torch.float32, device="cuda")


def tree(g, B, kids, depth):
    """parent [B], parents first, and each node's number among its siblings."""
    parent, nth, has, deep = [], [], [0] * (B + 1), [0] * (B + 1)
    for i in range(B):
        may = [r for r in range(i + 1) if has[r] < kids and deep[r] < depth]
        r = int(g.choice(may)) if may else i
        parent.append(r - 1)
        nth.append(has[r])
        has[r] += 1
        deep[i + 1] = deep[r] + 1
    return np.array(parent), np.array(nth)


def draw_tokens(g, parent, nth, draft, Td):
    """Children drawn from their rows without replacement."""
    token = np.full(len(parent), -1)
    for row in set(parent + 1):
        mine = np.flatnonzero(parent == row - 1)
        with np.errstate(divide="ignore"):
            order = np.argsort(-(draft[row].astype(np.float64) / Td - np.log(g.exponential(size=draft.shape[1]))), kind="stable")
        token[mine] = order[np.minimum(nth[mine], draft.shape[1] - 1)]
    return token


def problem(g, R, B, V, kids, depth, spread=2.0, noise=0.7, Td=None):
    """(parent, token, n, logits, draft) as numpy, logits as bf16 rounds them."""
    z = (g.standard_normal((R, B + 1, V)) * spread - 1.1 * np.log(1 + g.permutation(V)) + 15).astype(np.float32)
    d = (z + g.standard_normal(z.shape) * noise).astype(np.float32)
    z, d = (torch.from_numpy(x).to(BF16).float().numpy() for x in (z, d))
    n = g.integers(0, B + 1, R)
    n[0] = B
    par, tok = np.full((R, B), -1), np.full((R, B), -1)
    for r in range(R):
        p, nth = tree(g, B, kids, depth)
        k = int(n[r])
        par[r, :k] = p[:k]
        tok[r, :k] = draw_tokens(g, p[:k], nth[:k], d[r], 1.0 if Td is None else float(Td[r]))
    return par, tok, n, z, d


def check(par, tok, n, z, d, u, *, max_len=40, chain=False, types=(F32, F32), out=None, open_=0, **rules):
    """One call against the reference; rules: T, k, p, mp, Td [R] each."""
    R = len(n)
    if out is None:
        dev = lambda x, t: torch.from_numpy(x).to(t).cuda()  # noqa: E731
        out = run(par, tok, n, dev(z, types[0]), dev(d, types[1]), u, max_len=max_len, chain=chain, **rules)
    got = {k: host(v) for k, v in out.items()}
    near = 0
    for r in range(R):
        rule = {k: float(np.float32(v[r])) if k != "k" else int(v[r]) for k, v in rules.items()}
        nodes, t, prob, tol, close = ref.verify(None if chain else par[r], tok[r], int(n[r]), z[r], d[r], u[r], **rule)
        if close:
            near += 1
            continue
        assert got["len"][r] == len(nodes), (r, got["len"][r], nodes)
        want = (nodes + [-1] * max_len)[:max_len]
        assert got["nodes"][r].tolist() == want, (r, got["nodes"][r], want)
        assert got["bonus"][r] == t, (r, got["bonus"][r], t)
        assert abs(got["prob"][r] - prob) <= tol, (r, got["prob"][r], prob, tol)
    assert near <= open_ + 1 + 0.05 * R, near
    return out


def run(par, tok, n, z, d, u, *, max_len=40, chain=False, T=None, k=None, p=None, mp=None, Td=None):
    return dtl.verify(None if chain else cu(par), cu(tok), cu(n), z, d, f32(u), max_len=max_len,
                      temperature=None if T is None else f32(T), top_k=None if k is None else cu(k),
                      top_p=None if p is None else f32(p), min_p=None if mp is None else f32(mp),
                      draft_temperature=None if Td is None else f32(Td))


SIZES = [  # R, B, V, kids, depth
    (3, 1, 1, 1, 1), (4, 2, 2, 2, 2), (6, 5, 7, 3, 3), (20, 8, 500, 1, 8), (12, 30, 1000, 4, 6), (5, 64, 4097, 3, 8),
    (2, 16, 32000, 2, 8), (40, 4, 5001, 1, 4), (3, 12, 151936, 3, 5), (1, 1024, 40, 30, 6), (170, 6, 300, 2, 4),
]
MIX = [  # T, k, p, mp, Td
    dict(), dict(T=0.8, Td=0.8), dict(T=1.3, Td=0.6), dict(T=0.7, p=0.9, Td=0.7), dict(k=20, T=0.6), dict(k=1),
    dict(T=1.0, k=50, p=0.95, mp=0.02), dict(mp=0.1), dict(T=0.0), dict(p=0.0), dict(T=30.0, p=0.5, Td=20.0), dict(k=1000, T=2.0),
]


@pytest.mark.parametrize("mix", range(len(MIX)))
@pytest.mark.parametrize("size", range(len(SIZES)))
def test_sizes_and_settings(size, mix):
    R, B, V, kids, depth = SIZES[size]
    g = np.random.default_rng(100 * size + mix)
    rules = {k: np.full(R, v) for k, v in MIX[mix].items()}
    par, tok, n, z, d = problem(g, R, B, V, kids, depth, Td=rules.get("Td"))
    types = [(F32, F32), (BF16, BF16), (F32, BF16), (BF16, F32)][(size + mix) % 4]
    u = g.random((R, B + 1)).astype(np.float32)
    check(par, tok, n, z, d, u, types=types, chain=kids == 1 and mix % 2 == 0, **rules)


@pytest.mark.parametrize("types", [(F32, F32), (BF16, BF16), (F32, BF16), (BF16, F32)])
@pytest.mark.parametrize("shift", range(4))
def test_alignments_and_strides(types, shift):
    """Rows that start anywhere, draft rows without the last, padded strides."""
    g = np.random.default_rng(shift)
    R, B, V = 6, 7, 2003
    par, tok, n, z, d = problem(g, R, B, V, 1, B)
    u = g.random((R, B + 1)).astype(np.float32)

    def placed(x, t, pad, at):
        out = torch.full((R, x.shape[1] + 1, V + pad), float("nan"), dtype=t, device="cuda")
        out[:, :x.shape[1], at:at + V] = torch.from_numpy(x).to(t)
        return out[:, :x.shape[1], at:at + V]

    Z, D = placed(z, types[0], 5 + shift, shift), placed(d[:, :B], types[1], 8 - shift, 3 - shift)
    T = np.full(R, 0.9)
    out = run(par, tok, n, Z, D, u, T=T)
    check(par, tok, n, z, d, u, T=T, out=out)


def test_settings_of_each_request():
    g = np.random.default_rng(77)
    R, B, V = 60, 20, 3001
    rules = dict(T=g.choice([0.0, 0.5, 1.0, 1.7, float("nan")], R, p=[.15, .3, .3, .2, .05]), k=g.choice([0, 0, 1, 10, 5000], R),
                 p=g.choice([1.0, 0.95, 0.5, 2.0], R), mp=g.choice([0.0, 0.0, 0.05, 1.0], R), Td=g.choice([0.5, 1.0, -1.0], R))
    par, tok, n, z, d = problem(g, R, B, V, 3, 7, Td=np.where(rules["Td"] > 0, rules["Td"], 1.0))
    check(par, tok, n, z, d, g.random((R, B + 1)).astype(np.float32), **rules)


def test_tokens_that_cannot_have_been_drawn():
    """Tokens outside the vocabulary, the same token twice, tokens without
    probability under the draft, drafts without any, point masses."""
    g = np.random.default_rng(5)
    R, B, V = 40, 12, 64
    par, tok, n, z, d = problem(g, R, B, V, 4, 4)
    n[:] = B
    for r in range(R):
        kind = r % 8
        if kind == 0:
            tok[r, ::3] = g.choice([-1, V, -7, 1 << 30])
        elif kind == 1:
            tok[r] = tok[r, 0]
        elif kind == 2:
            d[r][:, tok[r, 0]] = -np.inf
        elif kind == 3:
            d[r] = -np.inf
        elif kind == 4:
            d[r] = -np.inf
            d[r][:, tok[r, 1]] = 3.0        # all of the draft's probability on one token
        elif kind == 5:
            d[r][:, 5] = np.nan
            z[r][:, 9] = np.nan
        elif kind == 6:
            d[r] = z[r]                     # the target's own distribution: the first is accepted
        elif kind == 7:
            z[r][:, ::2] = -np.inf          # half of the tokens are not allowed
    u = g.random((R, B + 1)).astype(np.float32)
    out = check(par, tok, n, z, d, u)
    lens = host(out["len"])
    assert (lens[3::8] == 0).all()
    assert (lens[6::8] > 0).all()


@pytest.mark.parametrize("types", [(F32, F32), (BF16, BF16)])
@pytest.mark.parametrize("rules", [dict(k=500), dict(k=40, p=0.9), dict(p=0.6), dict(p=0.97, mp=0.01), dict(k=1024, mp=0.001),
                                   dict(k=3000, p=0.9)])
def test_cuts_among_ties(types, rules):
    """Few different logits: a cut falls on one that thousands of tokens share, of
    which the first are kept; rows over several CTAs."""
    g = np.random.default_rng(13)
    R, B, V = 3, 5, 40000
    par, tok, n, z, d = problem(g, R, B, V, 2, 4)
    z = (np.round(z / 2) * 2).astype(np.float32)
    n[:] = B
    u = g.random((R, B + 1)).astype(np.float32)
    check(par, tok, n, z, d, u, types=types, **{k: np.full(R, v) for k, v in rules.items()})


@pytest.mark.parametrize("V, first", [(5003, 300), (5003, 5), (40007, 301), (40001, 7)])
def test_cut_within_one_logit(V, first):
    """All tokens but a few share a logit, and top-k keeps the first of them: from
    one to all but one, in rows that begin and end at odd places.  u close to 1
    draws the last one kept."""
    R = 8
    g = np.random.default_rng(V + first)
    z = np.full((R, 2, V), 6.5, np.float32)
    for r in range(R):
        z[r][:, g.permutation(V)[:first] if r % 2 else np.arange(first)] = 7.0
    d = np.zeros_like(z)
    k = first + np.array([1, 2, 700, V // 3, V // 2, V - first - 9, V - first - 2, V - first - 1])
    u = np.full((R, 2), 1 - 2.0 ** -24, np.float32)
    for types in ((BF16, BF16), (F32, BF16)):
        out = check(np.full((R, 1), -1), np.zeros((R, 1)), np.zeros(R, int), z, d, u, types=types, k=k)
        assert (host(out["bonus"])[::2] == k[::2] - 1).all()


@pytest.mark.parametrize("V", [7, 900, 20011])
def test_smallest_random_numbers(V):
    """u[0] down to the smallest fp32.  Weights off by 2^-44 of the largest leave the
    first tokens' running sums open by e = V 2^-43 (p_max + q_max) / N, 1e-9 at V = 20011:
    a mark u[0] below that may fall on any of the leading tokens that are together
    less, so the six draws up to 1e-9 may each be undecided."""
    g = np.random.default_rng(V)
    draws = np.array([2.0 ** -149, 1e-40, 1e-30, 1e-20, 2.0 ** -45, 1e-9, 2.0 ** -25, 2.0 ** -24, 3e-5, 1 - 2.0 ** -24], np.float32)
    R, B = len(draws), 3
    par, tok, n, z, d = problem(g, R, B, V, 1, 3)
    u = g.random((R, B + 1)).astype(np.float32)
    u[:, 0] = draws
    check(par, tok, n, z, d, u, chain=True, open_=6)
    check(par, tok, n, z, d, u, chain=True, types=(BF16, BF16), p=np.full(R, 0.9), open_=6)


def test_infinite_logits():
    g = np.random.default_rng(6)
    R, B, V = 24, 6, 300
    par, tok, n, z, d = problem(g, R, B, V, 2, 4)
    n[:] = B
    for r in range(R):
        if r % 4 == 0:
            z[r][:, g.integers(0, V, 5)] = np.inf
        elif r % 4 == 1:
            d[r][:, g.integers(0, V, 5)] = np.inf
        elif r % 4 == 2:
            z[r] = -np.inf
        else:
            z[r][:, tok[r, 0]] = np.inf
            d[r][:, tok[r, 0]] = np.inf
    u = g.random((R, B + 1)).astype(np.float32)
    for rules in (dict(), dict(T=np.full(R, 0.5), k=np.full(R, 3)), dict(p=np.full(R, 0.9)), dict(T=np.zeros(R))):
        out = check(par, tok, n, z, d, u, **rules)
        assert (host(out["bonus"])[2::4] == -1).all() and not host(out["prob"])[2::4].any()


def test_ends_of_the_random_numbers_and_short_lists():
    """u = 0 (every drawn token that the target can say is accepted) and at its
    largest; paths longer than max_len keep their first nodes; trees without
    nodes."""
    g = np.random.default_rng(8)
    R, B, V = 30, 9, 200
    par, tok, n, z, d = problem(g, R, B, V, 1, B)
    n[:] = np.where(np.arange(R) % 5 == 0, 0, B)
    u = np.where(np.arange(R)[:, None] % 2 == 0, 0.0, np.float32(1 - 2.0 ** -24)) * np.ones((R, B + 1), np.float32)
    u = u.astype(np.float32)
    out = check(par, tok, n, z, d, u, max_len=3)
    lens = host(out["len"])
    assert (lens[::2] > 3).any() and (lens[::5] == 0).all()


def test_rows_off_the_path_are_not_read():
    g = np.random.default_rng(9)
    R, B, V = 5, 20, 1000
    par, tok, n, z, d = problem(g, R, B, V, 3, 6)
    u = g.random((R, B + 1)).astype(np.float32)
    first = run(par, tok, n, torch.from_numpy(z).cuda(), torch.from_numpy(d).cuda(), u)
    for r in range(R):
        path = {0} | {int(x) + 1 for x in host(first["nodes"])[r] if x >= 0}
        for row in set(range(B + 1)) - path:
            z[r, row], d[r, row] = np.inf, -np.inf
    again = run(par, tok, n, torch.from_numpy(z).cuda(), torch.from_numpy(d).cuda(), u)
    assert all(torch.equal(first[k], again[k]) for k in first)


def test_a_request_does_not_depend_on_the_others():
    """One request alone (more CTAs to a row) and among many."""
    g = np.random.default_rng(10)
    R, B, V = 200, 6, 20011
    par, tok, n, z, d = problem(g, 4, B, V, 3, 4)
    rep = lambda x: np.concatenate([x] * (R // 4))  # noqa: E731
    u = g.random((4, B + 1)).astype(np.float32)
    T, p = np.full(R, 0.9), np.array([1.0, 0.9, 1.0, 0.8] * (R // 4))
    Z, D = torch.from_numpy(rep(z)).cuda(), torch.from_numpy(rep(d)).cuda()
    many = run(rep(par), rep(tok), rep(n), Z, D, rep(u), T=T, p=p)
    for r in range(4):
        one = run(par[r:r + 1], tok[r:r + 1], n[r:r + 1], Z[r:r + 1], D[r:r + 1], u[r:r + 1], T=T[:1], p=p[r:r + 1])
        for k in ("len", "nodes", "bonus"):
            assert (host(many[k])[r::4] == host(one[k])[0]).all(), k
        assert np.abs(host(many["prob"])[r::4] - host(one["prob"])[0]).max() <= 2.0 ** -23


@pytest.mark.parametrize("p", [None, 0.8])
def test_the_first_token_is_distributed_as_the_targets(p):
    """2^16 requests with children drawn from a draft that is far from the target:
    the frequencies of the first token of the result are the target's
    probabilities, within 5 standard deviations each."""
    g = np.random.default_rng(11)
    R, V, kids = 1 << 16, 8, 3
    z, d = g.standard_normal(V).astype(np.float32) * 1.5, g.standard_normal(V).astype(np.float32) * 1.5
    with np.errstate(divide="ignore"):
        tok = np.argsort(-(d.astype(np.float64) - np.log(g.exponential(size=(R, V)))), axis=1)[:, :kids]
    Z = torch.from_numpy(z).cuda().expand(R, kids + 1, V)
    D = torch.from_numpy(d).cuda().expand(R, kids + 1, V)
    u = g.random((R, kids + 1)).astype(np.float32)
    # (rows V apart in memory: the expanded tensors have no strides)
    out = run(np.full((R, kids), -1), tok, np.full(R, kids), Z.contiguous(), D.contiguous(), u,
              p=None if p is None else np.full(R, p))
    nodes, bonus = host(out["nodes"])[:, 0], host(out["bonus"])
    first = np.where(nodes >= 0, tok[np.arange(R), np.maximum(nodes, 0)], bonus)
    want = ref.target(z, 1.0, 0, 1.0 if p is None else p, 0.0)
    have = np.bincount(first, minlength=V) / R
    assert (np.abs(have - want) <= 5 * np.sqrt(want * (1 - want) / R)).all(), (have, want)
    # the first child alone is accepted with probability sum min(p, q)
    alone = np.minimum(want, ref.softmax(d, 1.0)).sum()
    assert (nodes >= 0).mean() >= alone - 5 * np.sqrt(alone / R)


def test_captured_and_on_another_stream():
    g = np.random.default_rng(12)
    R, B, V = 4, 6, 3000
    par, tok, n, z, d = problem(g, R, B, V, 2, 5)
    u = g.random((2, R, B + 1)).astype(np.float32)
    Z, D = torch.from_numpy(z).cuda(), torch.from_numpy(d).cuda()
    args = (cu(par), cu(tok), cu(n), Z, D)
    uu = f32(u[0])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    on_side = dtl.verify(*args, uu, max_len=6, stream=side)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = dtl.verify(*args, uu, max_len=6)
    for i in range(2):
        uu.copy_(f32(u[i]))
        graph.replay()
        torch.cuda.synchronize()
        check(par, tok, n, z, d, u[i], max_len=6, out=out)
        if i == 0:
            assert all(torch.equal(out[k], on_side[k]) for k in out)


def test_refusals():
    R, B, V = 2, 3, 50
    par, tok, n = cu(np.full((R, B), -1)), cu(np.zeros((R, B))), cu([3, 3])
    z, d, u = torch.zeros(R, B + 1, V, device="cuda"), torch.zeros(R, B, V, device="cuda"), f32(np.zeros((R, B + 1)))
    good = dict(parent=par, token=tok, n_out=n, logits=z, draft=d, u=u)
    for bad in (dict(parent=par[:1]), dict(token=tok.long()), dict(token=tok[0]), dict(n_out=cu([3])), dict(logits=z.half()),
                dict(logits=z[:, :B]), dict(draft=d[:, :B - 1]), dict(draft=d[..., :V - 1]), dict(u=u[:, :B]), dict(u=u.double()),
                dict(logits=z.cpu()), dict(logits=z.transpose(1, 2).contiguous().transpose(1, 2)), dict(max_len=0),
                dict(temperature=f32([1.0])), dict(top_k=f32([1, 1])), dict(logits=z[:1])):
        with pytest.raises((TypeError, ValueError)):
            dtl.verify(**{**good, "max_len": 4, **bad})
    big = torch.zeros(1, 2, (1 << 18) + 1, device="cuda")
    with pytest.raises(dtl.DartreeError):
        dtl.verify(None, cu([[1]]), cu([1]), big, big, f32([[0.5, 0.5]]), max_len=1)
    with pytest.raises(dtl.DartreeError):
        dtl.verify(None, cu(np.zeros((1, 1025))), cu([1]), torch.zeros(1, 1026, 4, device="cuda"),
                   torch.zeros(1, 1026, 4, device="cuda"), f32(np.zeros((1, 1026))), max_len=1)
