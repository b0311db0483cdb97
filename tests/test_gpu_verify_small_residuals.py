"""Verification where little is left of the target: residuals far below the rows'
sums, children of the smallest weights, uniform drafts, rows of one CTA.  All
against the definition in 64 bits."""
from __future__ import annotations

import numpy as np
import pytest
import torch

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
