"""Plain references of the paged 4-bit cache and of sampling, in 64 bits and
one element, token or page at a time (numpy; no code of the library)."""
from __future__ import annotations

import numpy as np

E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
E4M3 = np.array([(m / 8.0) * 2.0 ** -6 if e == 0 else (1 + m / 8.0) * 2.0 ** (e - 7)
                 for e in range(16) for m in range(8)][:127])


def nearest(x: np.ndarray, grid: np.ndarray) -> np.ndarray:
    """Index of the nearest grid point (ties to the even index), saturating."""
    x = np.minimum(x, grid[-1])
    hi = np.clip(np.searchsorted(grid, x), 1, len(grid) - 1)
    lo = hi - 1
    a, b = x - grid[lo], grid[hi] - x
    return np.where((a < b) | ((a == b) & (lo % 2 == 0)), lo, hi)


def quantise(x: np.ndarray, unit: float = 1.0):
    """codes [..., dh] and scale indices [..., dh/16] of x [..., dh] (fp64)."""
    y = np.where(np.isnan(x), 0.0, x) / unit
    y = y.reshape(*x.shape[:-1], x.shape[-1] // 16, 16)
    sc = nearest(np.abs(y).max(-1) / 6.0, E4M3)
    s = E4M3[sc][..., None]
    with np.errstate(divide="ignore", invalid="ignore"):
        q = np.where(s > 0, np.abs(y) / s, 0.0)
    code = nearest(q, E2M1) | (np.signbit(y) << 3)
    return code.reshape(x.shape).astype(np.uint8), sc.astype(np.uint8)


def values(code: np.ndarray, sc: np.ndarray, unit: float = 1.0) -> np.ndarray:
    v = E2M1[code & 7] * np.where(code & 8, -1.0, 1.0)
    return (v.reshape(*code.shape[:-1], code.shape[-1] // 16, 16) * E4M3[sc][..., None]).reshape(code.shape) * unit


def page_views(page: np.ndarray, P: int, Hkv: int, dh: int):
    """(key codes [Hkv, P, dh], key scales [Hkv, P, dh/16], value codes,
    value scales) of one page's bytes."""
    c = page.reshape(Hkv, -1)
    out, at = [], 0
    for _ in range(2):
        raw = c[:, at:at + P * dh // 2].reshape(Hkv, P, dh // 2)
        at += P * dh // 2
        code = np.empty((Hkv, P, dh), np.uint8)
        code[..., 0::2], code[..., 1::2] = raw & 15, raw >> 4
        out.append(code)
        out.append(c[:, at:at + P * dh // 16].reshape(Hkv, P, dh // 16))
        at += P * dh // 16
    return out


def token_values(pool_layer: np.ndarray, row: np.ndarray, pos: int, P: int, Hkv: int, dh: int,
                 ks: float = 1.0, vs: float = 1.0):
    """fp64 (k, v) [Hkv, dh] of one token."""
    kc, ksc, vc, vsc = page_views(pool_layer[row[pos // P]], P, Hkv, dh)
    t = pos % P
    return values(kc[:, t], ksc[:, t], ks), values(vc[:, t], vsc[:, t], vs)


def attention(q, K, V, see, scale):
    """q [n, Hq, dh], K, V [L, Hkv, dh], see [n, L] -> O [n, Hq, dh] (fp64)."""
    n, Hq, dh = q.shape
    g = Hq // K.shape[1] if K.shape[1] else 1
    O = np.zeros((n, Hq, dh))
    if K.shape[0] == 0:
        return O
    for h in range(Hq):
        z = np.where(see, scale * (q[:, h] @ K[:, h // g].T), -np.inf)
        top = z.max(1, keepdims=True)
        w = np.exp(z - np.where(np.isinf(top), 0.0, top))
        tot = w.sum(1, keepdims=True)
        O[:, h] = (w @ V[:, h // g]) / np.where(tot > 0, tot, 1.0)
    return O


class Pages:
    """The page operations, one row and page at a time."""

    def __init__(self, pool, refs, table, lens, P):
        self.pool, self.refs, self.table, self.lens, self.P = (pool.copy(), refs.copy(),
                                                               table.copy(), lens.copy(), P)

    def held(self, r):
        n = 0
        while n < self.table.shape[1] and self.table[r, n] >= 0:
            n += 1
        return n

    def reserve(self, want):
        R, width = self.table.shape
        ok, taken, out = np.zeros(R, np.int32), 0, False
        free = int((self.refs == 0).sum())
        for r in range(R):
            if self.lens[r] < 0 or want[r] < 0:
                continue
            need = -(-(int(self.lens[r]) + int(want[r])) // self.P)
            if need > width:
                continue
            lack = max(0, need - self.held(r))
            out = out or taken + lack > free
            if lack and out:
                continue
            ok[r] = 1
            taken += lack
            for _ in range(lack):
                page = int(np.flatnonzero(self.refs == 0)[0])
                self.table[r, self.held(r)] = page
                self.refs[page] = 1
        return ok

    def fork(self, src, dst):
        R, width = self.table.shape
        ok = np.zeros(len(src), np.int32)
        empty = [0 <= d < R and self.held(d) == 0 for d in dst]
        out = False
        for i, (s, d) in enumerate(zip(src, dst)):
            if not (0 <= s < R and 0 <= d < R) or d in src or d in dst[:i] or not empty[i]:
                continue
            n = int(self.lens[s])
            if n < 0 or -(-n // self.P) > self.held(s):
                continue
            if n % self.P:
                free = np.flatnonzero(self.refs == 0)
                out = out or len(free) == 0
                if out:
                    continue
            ok[i] = 1
            whole = n // self.P
            for j in range(whole):
                self.table[d, j] = self.table[s, j]
                self.refs[self.table[s, j]] += 1
            if n % self.P:
                page = int(free[0])
                self.refs[page] = 1
                self.table[d, whole] = page
                self.pool[:, page] = self.pool[:, self.table[s, whole]]
            self.lens[d] = n
        return ok

    def release(self, rows, keep):
        R, width = self.table.shape
        for r, k in zip(rows, keep):
            if not 0 <= r < R or k < 0:
                continue
            for j in range(-(-int(k) // self.P), width):
                if self.table[r, j] >= 0:
                    self.refs[self.table[r, j]] -= 1
                    self.table[r, j] = -1
            self.lens[r] = min(self.lens[r], k)

    def commit(self, nodes, length, extra, Hkv, dh):
        R, most = nodes.shape
        P = self.P
        for r in range(R):
            if self.lens[r] < 0:
                continue
            m, n = max(0, min(int(length[r]), most)), int(self.lens[r])
            path = nodes[r, :m]
            pos = [n + int(x) for x in path] + [n + k for k in range(m)]
            if (m and path[0] < 0) or (np.diff(path) <= 0).any() or any(
                    p // P >= self.held(r) for p in pos):
                continue
            for k in range(m):
                src, dst = n + int(path[k]), n + k
                for layer in range(self.pool.shape[0]):
                    a = self.pool[layer, self.table[r, src // P]].reshape(Hkv, -1)
                    b = self.pool[layer, self.table[r, dst // P]].reshape(Hkv, -1)
                    at = 0
                    for unit in (dh // 2, dh // 16) * 2:
                        sa, da = at + (src % P) * unit, at + (dst % P) * unit
                        b[:, da:da + unit] = a[:, sa:sa + unit].copy()
                        at += P * unit
            self.lens[r] = n + m + extra


def sample_row(l, T, k, p, mp, u):
    """(token, prob, margin) of one row: margin is how far the nearest border
    of any decision lies from its value, relative to the whole."""
    l = np.where(np.isnan(l), -np.inf, l.astype(np.float64))
    top = l.max()
    if top == -np.inf:
        return -1, 0.0, 1.0
    if not T > 0:
        return int(np.argmax(l)), 1.0, 1.0
    with np.errstate(invalid="ignore"):
        d = np.where(l == top, 0.0, l - top)
    w = np.exp(d / T)
    order = np.lexsort((np.arange(len(l)), -l))
    ws = w[order]
    n, margin = len(l), 1.0
    if 1 <= k < n:
        n = k
    if mp > 0:
        mp = min(mp, 1.0)
        margin = min(margin, np.abs(ws[ws != 1.0] - mp).min(initial=1.0) if mp < 1 else 1.0)
        n = min(n, int((ws >= mp).sum()))
    if p < 1:
        cum = np.cumsum(ws[:n])
        at = p * cum[-1]
        margin = min(margin, np.abs(cum[:-1] - at).min(initial=1.0) / cum[-1])
        n = min(n, int((cum < at).sum()) + 1) if p > 0 else 1
    kept = np.sort(order[:n])
    cum = np.cumsum(w[kept])
    t = u * cum[-1]
    margin = min(margin, np.abs(cum[:-1] - t).min(initial=1.0) / cum[-1])
    j = min(int((cum <= t).sum()), n - 1)
    return int(kept[j]), float(w[kept[j]] / cum[-1]), float(margin)
