"""Sampling on the GPU against the definition in 64 bits, row by row."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from speculative_decoding_draft_06_gb300 import dartree as dtl
from tests import cache_ref as ref

pytestmark = pytest.mark.gpu



def f32(x):
    return torch.tensor(x, dtype=torch.float32, device="cuda")


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def check(logits, u, per, T, k, p, m, exact=False):
    """One call against the reference, every row.  prob is w / total rounded
    to fp32 (2^-24), the weights being off by 2^-44 of the largest at most:
    2^-25 of a weight above 2^-19; below, the difference is absolute.  exact:
    the weights are whole numbers on both sides, and so are values on a
    border."""
    n = -(-len(u) // per)
    got = dtl.sample(logits, torch.from_numpy(u).cuda(), rows_per_req=per, temperature=None if T is None else f32(T),
                     top_k=None if k is None else i32(k), top_p=None if p is None else f32(p),
                     min_p=None if m is None else f32(m))
    tok, prob = got["token"].cpu().numpy(), got["prob"].cpu().numpy()
    l = logits.float().cpu().numpy()
    near = 0
    f = lambda a, d, r: d if a is None else float(np.float32(a[r]))  # noqa: E731
    for i in range(len(u)):
        r = i // per
        assert r < n
        t, q, margin = ref.sample_row(l[i], f(T, 1.0, r), int(f(k, 0, r)), f(p, 1.0, r), f(m, 0.0, r), float(u[i]))
        if margin < 2.0 ** -40 and not exact:      # the border is where the value is: both sides' last bits decide
            near += 1
            continue
        assert tok[i] == t, (i, tok[i], t, margin)
        assert abs(prob[i] - q) <= 2.0 ** -23 * q + 2.0 ** -43, (i, prob[i], q)
    assert near <= 0.02 * len(u) + 1
    return tok, prob


MIX = [("full", None, None, None, None), ("temperature", [0.3], None, None, None), ("hot", [50.0], None, [0.9], None),
       ("k1", None, [1], None, None), ("k7", [0.8], [7], None, None), ("k1000", [1.0], [1000], [0.99], None),
       ("p", [0.7], None, [0.9], None), ("p small", None, None, [1e-6], None), ("p0", None, None, [0.0], None),
       ("m", [1.0], None, None, [0.05]), ("m1", None, None, None, [1.0]), ("all", [0.9], [50], [0.95], [0.02]),
       ("m p", [1.2], None, [0.8], [0.01]), ("greedy", [0.0], [5], [0.5], None), ("huge k", None, [10 ** 9], [1.0], [0.0]),
       ("negative", None, [-3], [2.0], [-1.0])]


@pytest.mark.parametrize("V", [1, 2, 31, 1000, 4097, 32000, 151936])
@pytest.mark.parametrize("mix", range(len(MIX)))
def test_every_setting(V, mix):
    """fp32 and bf16 logits of a vocabulary's usual shape, padding masked."""
    _, T, k, p, m = MIX[mix]
    g = np.random.default_rng(V + mix)
    rows = 5 if V > 5000 else 24
    x = g.standard_normal((rows, V)) * 2 - 1.1 * np.log(1 + g.permutation(V))[None] + 15
    if V > 30:
        x[:, -V // 50:] = -np.inf
        x[1, g.random(V) < 0.99] = -np.inf
    u = g.random(rows).astype(np.float32)
    for dt in (torch.float32, torch.bfloat16):
        check(torch.from_numpy(x).to(dt).cuda(), u, rows, T, k, p, m)


def test_settings_of_each_request_and_strides():
    g = np.random.default_rng(3)
    R, per, V = 9, 13, 5000
    x = torch.from_numpy(g.standard_normal((R * per - 4, V + 3)) * 3).float().cuda()[:, 1:V + 1]
    assert x.stride(0) == V + 3
    u = g.random(R * per - 4).astype(np.float32)       # (the last request has fewer rows)
    check(x, u, per, g.choice([0.0, 0.5, 1.0, 2.0], R), g.choice([0, 1, 10, 300], R), g.choice([1.0, 0.9, 0.3], R),
          g.choice([0.0, 0.1], R))
    check(x[:, :777], u, 1, g.choice([0.0, 0.5, 1.0, 2.0], len(u)), None, g.choice([1.0, 0.9, 0.3], len(u)), None)


@pytest.mark.parametrize("V", [7, 3000, 100000])
def test_ties(V):
    """Equal logits: the order is the index's; large classes of equal keys."""
    g = np.random.default_rng(V)
    for levels in (1, 2, 5):
        x = g.integers(0, levels, (6, V)).astype(np.float32)
        u = g.random(6).astype(np.float32)
        for k, p in ((None, None), ([V // 2 + 1], None), (None, [0.37]), ([V - 1], [0.61]), ([1], None)):
            check(torch.from_numpy(x).cuda(), u, 6, None, k, p, None)


@pytest.mark.parametrize("V", [40, 5000, 70001])
@pytest.mark.parametrize("centre,spread", [(0.0, 0.5), (12.0, 3.0), (-8.0, 2.0), (-0.01, 0.005), (300.0, 100.0)])
def test_bf16_cuts_among_ties(V, centre, spread):
    """Top-k and top-p of whole rows that fall among many equal logits, rows
    that start at any address."""
    g = np.random.default_rng(V)
    x = torch.from_numpy(g.standard_normal((4, V + 5)) * spread + centre).to(torch.bfloat16)
    x[1] = (x[1].float() * 4).round().to(torch.bfloat16) / 4
    x[2, ::7] = x[2, 3]
    x[3, ::5] = float("nan")
    x[3, 1::5] = -float("inf")
    u = g.random(4).astype(np.float32)
    for off in (0, 1, 5):
        t = x.cuda()[:, off:off + V]
        for T in (1.0, 5.0):
            for k, p in ((V // 3, 1.0), (V - 2, 0.97), (V // 2, 0.6), (0, 0.9), (0, 0.999), (0, 1.0)):
                check(t, u, 4, [T], [k], [p], None)


@pytest.mark.parametrize("V", [9, 20000, 100000])
def test_the_two_zeros_are_equal(V):
    g = np.random.default_rng(V)
    x = np.where(g.random((6, V)) < 0.5, np.float32(-0.0), np.float32(0.0))
    x[3:, V // 2:] = -1.0
    u = g.random(6).astype(np.float32)
    for dt in (torch.float32, torch.bfloat16):
        t = torch.from_numpy(x).to(dt).cuda()
        for T, k, p in ((0.0, 0, 1.0), (1.0, 1, 1.0), (1.0, V // 3, 1.0), (1.0, 0, 0.4), (0.7, 5, 0.5)):
            check(t, u, 6, [T], [k], [p], None)


@pytest.mark.parametrize("V", [50, 3001, 60000])
def test_extreme_settings(V):
    """Temperatures from the smallest to infinity; NaN settings cut nothing (a
    temperature: the largest logit)."""
    g = np.random.default_rng(V)
    x = torch.from_numpy(g.standard_normal((5, V)).astype(np.float32) * 3)
    u = g.random(5).astype(np.float32)
    big = float(np.finfo(np.float32).max)
    for t in (x.cuda(), x.to(torch.bfloat16).cuda()):
        for T in (float("inf"), big, 1e30, 1e5, 1e-5, 1e-30, 1e-38):
            for k, p, m in ((0, 1.0, 0.0), (7, 1.0, 0.0), (0, 0.5, 0.0), (0, 1.0, 0.5), (V // 2, 0.9, 0.1)):
                check(t, u, 5, [T], [k], [p], [m], exact=T >= 1e30)  # (there all weights are 1)
        nan = dtl.sample(t, torch.from_numpy(u).cuda(), rows_per_req=5, top_p=f32([float("nan")]), min_p=f32([float("nan")]))
        none = dtl.sample(t, torch.from_numpy(u).cuda())
        assert torch.equal(nan["token"], none["token"]) and torch.equal(nan["prob"], none["prob"])
        cold = dtl.sample(t, torch.from_numpy(u).cuda(), rows_per_req=5, temperature=f32([float("nan")]))
        assert torch.equal(cold["token"], t.float().argmax(1).int())


def test_exact_borders():
    """Equal weights make the borders whole numbers: u and top_p that fall on
    them are decided by 'exceeds u' and 'at least top_p'."""
    V = 8
    x = torch.zeros(9, V, device="cuda")
    u = np.array([i / 8 for i in range(8)] + [np.nextafter(np.float32(1), np.float32(0))], np.float32)
    tok = dtl.sample(x, torch.from_numpy(u).cuda())["token"].cpu().tolist()
    assert tok == [0, 1, 2, 3, 4, 5, 6, 7, 7]
    for p, n in ((0.125, 1), (0.25, 2), (0.5, 4), (0.5000001, 5), (0.875, 7)):
        last = dtl.sample(x, torch.full((9,), 0.99999, device="cuda"), rows_per_req=9, top_p=f32([p]))
        assert last["token"].cpu().tolist() == [n - 1] * 9
        assert np.allclose(last["prob"].cpu().numpy(), 1 / n, rtol=2.0 ** -23)
    # u outside [0, 1)
    odd = dtl.sample(x[:4], f32([1.0, -0.5, 7.0, float("nan")]))["token"].cpu().tolist()
    assert odd == [7, 0, 7, 0]


def test_infinities_nan_and_empty_rows():
    inf, nan = float("inf"), float("nan")
    x = torch.zeros(8, 100, device="cuda")
    x[0] = -inf
    x[1] = nan
    x[2] = nan
    x[2, 40] = -5.0
    x[3, 10], x[3, 20] = inf, inf
    x[4] = -inf
    x[4, 99] = -3.4e38
    x[5] = -3.4028234663852886e38
    x[5, 7] = 3.4028234663852886e38
    x[6, ::2] = nan
    x[7, 50] = inf
    for T in (1.0, 0.0, 0.01, inf):
        for p in (None, f32([0.9])):
            out = dtl.sample(x, torch.full((8,), 0.75, device="cuda"), rows_per_req=8, temperature=f32([T]), top_p=p)
            tok, prob = out["token"].cpu().tolist(), out["prob"].cpu().tolist()
            assert tok[0] == tok[1] == -1 and prob[0] == prob[1] == 0.0
            assert tok[2] == 40 and prob[2] == 1.0
            assert tok[3] == (10 if T == 0.0 else 20)
            assert tok[4] == 99 and prob[4] == 1.0
            assert tok[5] == 7 or T == inf
            assert tok[6] % 2 == 1 if T != 0.0 else tok[6] == 1
            assert tok[7] == 50


def test_results_do_not_depend_on_the_launch():
    """A row alone, among few and among many rows (other cluster sizes), and
    in a replayed graph: the same tokens and probabilities, bit for bit."""
    g = np.random.default_rng(9)
    x = torch.from_numpy(g.standard_normal((400, 20000)) * 2).float().cuda()
    u = torch.from_numpy(g.random(400).astype(np.float32)).cuda()
    kw = dict(rows_per_req=400, temperature=f32([0.9]), top_k=i32([3000]), top_p=f32([0.97]))
    many = dtl.sample(x, u, **kw)
    for n in (1, 20, 100):
        few = dtl.sample(x[:n], u[:n], **kw)
        assert torch.equal(few["token"], many["token"][:n]) and torch.equal(few["prob"], many["prob"][:n])
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        out = dtl.sample(x, u, **kw)
    u.copy_(torch.flip(u, [0]))
    gr.replay()
    again = dtl.sample(x, u, **kw)
    torch.cuda.synchronize()
    assert torch.equal(out["token"], again["token"])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    other = dtl.sample(x, u, stream=s, **kw)
    s.synchronize()
    assert torch.equal(other["token"], again["token"])


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("shift", [-6.0, 6.0])
def test_rows_whose_spread_out_units_mislead(bf16, shift):
    """256 evenly spread units of 16 bytes lie far below or above the rest of
    the row: a bound that is taken from them lets nearly all tokens pass, or
    almost none."""
    V, rows = 40008, 4
    g = np.random.default_rng(5)
    x = g.standard_normal((rows, V)).astype(np.float32)
    per = 8 if bf16 else 4
    units = V // per
    for t in range(256):
        at = t * units // 256 * per
        x[:, at:at + per] += shift
    x = torch.from_numpy(x).to(torch.bfloat16 if bf16 else torch.float32).cuda()
    u = g.random(rows).astype(np.float32)
    for T, k, p, m in ((1.0, 20, 1.0, 0.0), (1.0, 1000, 1.0, 0.0), (0.5, 1000, 0.9, 0.0), (1.0, 2500, 1.0, 0.0),
                       (1.0, 2500, 0.8, 0.01), (1.0, 9000, 0.999, 0.0), (1.0, 30000, 1.0, 0.0), (0.3, 0, 0.5, 0.0),
                       (1.0, 0, 0.99, 0.0), (1.0, 0, 1.0, 0.2), (1.0, 0, 0.9, 1e-4), (0.0, 0, 1.0, 0.0), (3.0, 0, 0.3, 0.0)):
        check(x, u, rows, [T], [k], [p], [m])


@pytest.mark.parametrize("V", [300, 60000])
@pytest.mark.parametrize("low,high", [(-0.3, 0.3), (-30.0, -0.05), (-9.0, 5.0), (1e-38, 1e-30), (-3e4, -2e4), (-1.0, 0.0)])
def test_bf16_logits_of_all_sizes(low, high, V):
    """Whole rows of bf16 logits, most of them on either side of zero, at
    zero, subnormal or far from it."""
    g = np.random.default_rng(V)
    x = torch.from_numpy(g.uniform(low, high, (4, V))).to(torch.bfloat16)
    x[1, ::3] = 0.0
    x[1, 1::3] = -0.0
    x[2, ::2] = high
    u = g.random(4).astype(np.float32)
    for T in (1.0, 0.1, 20.0):
        for p in (1.0, 0.95, 0.4):
            check(x.cuda(), u, 4, [T], None, [p], None)


@pytest.mark.parametrize("bf16", [False, True])
def test_the_largest_vocabulary(bf16):
    """2^18 tokens: all equal (sums of 2^62), two values, the usual shape, and
    the type's extremes."""
    V = 1 << 18
    g = np.random.default_rng(18)
    x = np.zeros((5, V), np.float32)
    x[1] = g.integers(0, 2, V)
    x[2] = g.standard_normal(V) * 2 - 1.1 * np.log(1 + g.permutation(V)) + 15
    x[3] = g.uniform(-3.3e38, -1e38, V)
    x[4] = g.uniform(1e38, 3.3e38, V)
    t = torch.from_numpy(x).to(torch.bfloat16 if bf16 else torch.float32).cuda()
    u = np.array([0.3, 0.999, 0.5, 0.2, 0.8], np.float32)
    for T, k, p in ((1.0, 0, 1.0), (1.0, V - 1, 0.7), (2.0, 0, 0.97), (1.0, 5, 1.0), (0.0, 0, 1.0)):
        check(t, u, 5, [T], [k], [p], None)
    assert dtl.sample(t[:1], torch.tensor([1.0], device="cuda"))["token"].item() == V - 1


@pytest.mark.parametrize("R,per,last", [(300, 3, 3), (300, 3, 1), (1024, 1, 1), (1030, 1, 1), (33, 2, 2)])
def test_many_requests_of_all_kinds(R, per, last):
    """Rows that need their whole row's weights among rows that do not."""
    g = np.random.default_rng(R)
    V, rows = 700, R * per - (per - last)
    x = torch.from_numpy(g.standard_normal((rows, V)).astype(np.float32) * 2).cuda()
    u = g.random(rows).astype(np.float32)
    check(x, u, per, g.choice([0.0, 0.5, 1.0, 2.0], R), g.choice([0, 0, 1, 10, 300], R),
          g.choice([1.0, 0.9, 0.3], R), g.choice([0.0, 0.0, 0.1], R))


def test_draws_follow_the_distribution():
    """40000 draws of one row: each kept token's count within 6 standard
    deviations of its share, none of the others."""
    g = np.random.default_rng(1)
    l = g.standard_normal(50).astype(np.float32) * 2
    n = 40000
    x = torch.from_numpy(l).cuda().expand(n, 50).contiguous()
    u = torch.from_numpy(g.random(n).astype(np.float32)).cuda()
    tok = dtl.sample(x, u, rows_per_req=n, top_k=i32([12]))["token"].cpu().numpy()
    w = np.exp(l.astype(np.float64))
    w[np.argsort(-l)[12:]] = 0
    w /= w.sum()
    cnt = np.bincount(tok, minlength=50)
    assert (np.abs(cnt - n * w) <= 6 * np.sqrt(n * w * (1 - w)) + 1e-9).all()


def test_binding_refuses_bad_tensors():
    x, u = torch.zeros(4, 10, device="cuda"), torch.zeros(4, device="cuda")
    for bad in (x.half(), x.cpu()):
        with pytest.raises(TypeError):
            dtl.sample(bad, u)
    with pytest.raises(ValueError):
        dtl.sample(x.t().contiguous().t(), u)
    with pytest.raises(ValueError):
        dtl.sample(x, u[:3])
    with pytest.raises(ValueError):
        dtl.sample(x, u, rows_per_req=2, temperature=f32([1.0]))
    with pytest.raises(TypeError):
        dtl.sample(x, u, top_k=f32([1.0] * 4))
