"""Verification where little is left of the target: residuals far below the rows'
sums, children of the smallest weights, uniform drafts, rows of one CTA.  All
against the definition in 64 bits."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from tests import verify_ref as ref
from tests.test_gpu_cache import host
from tests.test_gpu_verify_draft import BF16, F32, check, run

pytestmark = pytest.mark.gpu

LN2 = float(np.log(2.0))


@pytest.mark.parametrize("bits", [30.0, 43.9, 44.1, 44.5, 44.9, 45.2])
@pytest.mark.parametrize("types", [(F32, F32), (F32, BF16)])
def test_the_first_child_has_the_smallest_weight(bits, types):
    """The first child's weight under the draft is 2^-bits of the largest, from 2^-45
    on one unit of 2^-44: with the target's p = 0.25 it is accepted, whatever top-p
    says of the second, the draft's likeliest.  Below that it cannot have been drawn."""
    R, V = 6, 40
    z = np.full((R, 3, V), -6.0, np.float32)
    z[:, :, 3], z[:, :, 7] = 1.0, 0.0
    d = np.full((R, 3, V), -3.0, np.float32)
    d[:, :, 3] = bits * LN2 / 2
    d[:, :, 7] = np.float32(-bits * LN2 / 2)
    d = torch.from_numpy(d).to(types[1]).float().numpy()
    drawn = (d[0, 0, 3].astype(np.float64) - d[0, 0, 7]) / LN2 < 45
    tok, par = np.tile([7, 3], (R, 1)), np.full((R, 2), -1)
    u = np.zeros((R, 3), np.float32)
    u[:, 1] = 0.5
    u[:, 0] = np.linspace(0.0, 0.9, R)
    for rules in (dict(p=np.full(R, 0.98)), dict(), dict(p=np.full(R, 0.98), k=np.full(R, 30)), dict(p=np.full(R, 0.98), mp=np.full(R, 1e-3))):
        out = check(par, tok, np.full(R, 2), z, d, u, types=types, **rules)
        assert (host(out["nodes"])[:, 0] == (0 if drawn else 1)).all(), rules


@pytest.mark.parametrize("V", [7, 300, 5003])
@pytest.mark.parametrize("types", [(F32, F32), (BF16, BF16), (F32, BF16), (BF16, F32)])
def test_infinite_temperatures(V, types):
    """A draft (or a target) of infinite temperature is uniform over its tokens above
    -inf: the same as equal logits there."""
    g = np.random.default_rng(V)
    R, B = 20, 3
    par, n = np.tile([-1, -1, 0], (R, 1)), np.full(R, B)
    z = torch.from_numpy((2 * g.standard_normal((R, B + 1, V))).astype(np.float32)).to(BF16).float().numpy()
    d = torch.from_numpy((2 * g.standard_normal((R, B + 1, V))).astype(np.float32)).to(BF16).float().numpy()
    gone = g.random((R, B + 1, V)) < 0.4
    gone[:, :, 0] = False
    flat = np.where(gone, -np.inf, 0.0).astype(np.float32)
    tok = np.stack([g.choice(np.flatnonzero(~gone[r, 0]), 3, replace=V < 8) for r in range(R)])
    u = g.random((R, B + 1)).astype(np.float32)
    inf = np.full(R, np.inf)

    def dev(x, t):
        return torch.from_numpy(x.astype(np.float32)).to(t).cuda()

    out = run(par, tok, n, dev(z, types[0]), dev(np.where(gone, -np.inf, d), types[1]), u, Td=inf)
    check(par, tok, n, z, flat, u, out=out)
    out = run(par, tok, n, dev(np.where(gone, -np.inf, z), types[0]), dev(d, types[1]), u, T=inf)
    check(par, tok, n, flat, d, u, out=out)


def agreeing(g, R, V, bits, rows):
    """A target that is its draft but for one token x, whose weight under the draft
    is 2^-bits of the largest.  (z, d, x, the draft's second)"""
    z = np.repeat((g.standard_normal((R, 1, V)) * 2).astype(np.float32), rows, 1)
    order = np.argsort(-z[:, 0], axis=1)
    x, y = order[:, V // 2], order[:, 1]
    for r in range(R):
        z[r, :, x[r]] = z[r, 0].max() - np.float32(bits * LN2)
    return z, z.copy(), x, y


def undecided(R, V, bits):
    """How many of R results may be undecided: a partial sum of a residual of N = 2^-bits
    p_max or more is off by e = V 2^-43 (p_max + q_max) (1 + A) / N <= V 2^(bits - 41), and V of
    them have a mark within 2 e on either side."""
    return int(R * min(1.0, 4 * V * V * 2.0 ** (bits - 41)))


def second(z, x2, bits):
    """The bits of N behind two rejections: p is q (1 + N) but for the first child, so
    max(p - A q, 0) sums up to N q(x2), x2 the second."""
    p = np.array([ref.softmax(row[0], 1.0)[x] / ref.softmax(row[0], 1.0).max() for row, x in zip(z, x2)])
    return bits - float(np.log2(p.min()))


AGREE = [(64, 12), (64, 16), (64, 19), (64, 22), (500, 12), (500, 15), (500, 18), (3000, 12), (3000, 14)]


@pytest.mark.parametrize("V, bits", AGREE)
@pytest.mark.parametrize("types", [(F32, F32), (F32, BF16)])
def test_a_sibling_after_a_small_residual(V, bits, types):
    """x is rejected and N = sum max(p - q, 0), half of q(x), is spread over all other
    tokens in proportion: the next child's p - q is N q of it, accepted at any u
    below about 1."""
    g = np.random.default_rng(1000 * V + bits)
    R = 100
    z, d, x, y = agreeing(g, R, V, bits, 3)
    if types[1] is BF16:
        z, d = (torch.from_numpy(a).to(BF16).float().numpy() for a in (z, d))
    for r in range(R):
        z[r, :, x[r]] -= np.float32(0.75)
    u = np.stack([g.random(R), np.full(R, 0.9), g.random(R)], 1).astype(np.float32)
    out = check(np.full((R, 2), -1), np.stack([x, y], 1), np.full(R, 2), z, d, u, types=types, open_=undecided(R, V, bits))
    assert (host(out["nodes"])[:, 0] == 1).mean() > 0.9


@pytest.mark.parametrize("V, bits", AGREE + [(64, 24)])
@pytest.mark.parametrize("child", [1, 2])
def test_a_draw_from_a_small_residual(V, bits, child):
    """The target cannot say x, the only drafted token: its own is drawn from the other
    tokens in proportion to p.  With a second child that it cannot say either, from
    what is left behind two rejections."""
    g = np.random.default_rng(2000 * V + 10 * bits + child)
    R = 100
    z, d, x, y = agreeing(g, R, V, bits, 3)
    tok = np.stack([x, np.argsort(-z[:, 0], axis=1)[:, V // 2 + 1]], 1)
    for r in range(R):
        z[r, :, tok[r, :child]] = -np.inf
    u = np.stack([g.random(R), g.random(R), g.random(R)], 1).astype(np.float32)
    if child == 2:
        bits = second(d, tok[:, 1], bits)
    check(np.full((R, 2), -1), tok, np.full(R, child), z, d, u, open_=undecided(R, V, bits))


@pytest.mark.parametrize("V", [12, 300, 20011])
@pytest.mark.parametrize("types", [(F32, F32), (BF16, BF16)])
def test_two_logits_changed_places(V, types):
    """The target has the draft's logits with those of x and y exchanged: p = A q for
    all other tokens, exactly, and nothing but y is left behind a rejected x."""
    g = np.random.default_rng(V)
    R = 30
    d = torch.from_numpy((g.standard_normal((R, 1, V)) * 2).astype(np.float32)).to(types[0]).float().numpy().repeat(2, 1)
    z, x, y = d.copy(), np.zeros(R, int), np.zeros(R, int)
    for r in range(R):
        order = np.argsort(-d[r, 0])
        x[r], y[r] = order[g.integers(0, 3)], order[g.integers(3, min(V, 40))]
        z[r, :, x[r]], z[r, :, y[r]] = d[r, 0, y[r]], d[r, 0, x[r]]
    u = np.stack([g.random(R), np.full(R, 1 - 2.0 ** -24)], 1).astype(np.float32)
    out = check(np.full((R, 1), -1), x[:, None], np.ones(R, int), z, d, u, types=types)
    rejected = host(out["len"]) == 0
    assert rejected.sum() > R // 2 and (host(out["bonus"])[rejected] == y[rejected]).all()


@pytest.mark.parametrize("types", [(F32, F32), (BF16, BF16)])
def test_one_large_logit_per_thread_and_a_flat_tail(types):
    """More requests than share a row between CTAs, at the largest vocabulary: a thread
    sums 512 tokens, a large one and 511 below half a unit of its last place.  The
    second child's u lies around what p, q and N = sum max(p - q, 0) accept, down
    to 2^-20 of it."""
    R, V = 160, 1 << 18
    g = np.random.default_rng(1)
    z = np.full(V, np.float32(-24.25 * LN2), np.float32)
    first = (np.arange(16)[:, None] * (V // 16) + np.arange(32)[None, :] * (4 if types[0] is F32 else 8)).ravel()
    z[first] = 0.0
    d = np.full(V, np.float32(-18 * LN2), np.float32)
    x, y = int(first[77]), int(first[300])
    z[x] = -20.0                     # the draft's likeliest, hardly the target's
    d[x], d[y] = 0.0, -6.4
    z, d = (torch.from_numpy(a).to(BF16).float().numpy() for a in (z, d))
    p, q = ref.target(z, 1.0, 0, 1.0, 0.0), ref.softmax(d, 1.0)
    N, Z = np.maximum(p - q, 0.0).sum(), 1.0 - q[x]
    edge = (p[y] - q[y]) / (N / Z * q[y])
    assert 0.3 < edge < 0.9
    off = np.concatenate([2.0 ** -np.arange(8, 21), -2.0 ** -np.arange(8, 21)])
    u = np.zeros((R, 3), np.float32)
    u[:, 1] = 0.9
    u[:, 2] = edge * (1 + np.resize(off, R))
    u[:, 0] = g.random(R)
    # (one request's three rows, the same for all requests)
    rows = [torch.from_numpy(np.tile(a, (1, 3, 1))).to(t).cuda().expand(R, 3, V) for a, t in ((z, types[0]), (d, types[1]))]
    par, tok, n = np.full((R, 2), -1), np.tile([x, y], (R, 1)), np.full(R, 2)
    out = run(par, tok, n, rows[0], rows[1], u)
    accepted = host(out["nodes"])[:, 0] == 1
    want = u[:, 2].astype(np.float64) * (N / Z) * q[y] < p[y] - q[y]
    assert (accepted == want).all(), np.flatnonzero(accepted != want)
    assert want.any() and not want.all()
