"""The verification of drafted tokens, one request at a time in 64 bits: the
residuals are made one after the other (no code of the library)."""
from __future__ import annotations

import numpy as np


def target(l, T, k, p, mp):
    """The target's probabilities after the cuts (None: no token)."""
    l = np.where(np.isnan(l), -np.inf, l.astype(np.float64))
    top = l.max()
    if top == -np.inf:
        return None
    with np.errstate(invalid="ignore"):
        w = np.exp(np.where(l == top, 0.0, l - top) / T)
    order = np.lexsort((np.arange(len(l)), -l))
    n = len(l)
    if 1 <= k < n:
        n = k
    if mp > 0:
        n = min(n, int((w[order] >= min(mp, 1.0)).sum()))
    if p < 1:
        cum = np.cumsum(w[order][:n])
        n = min(n, int((cum < p * cum[-1]).sum()) + 1) if p > 0 else 1
    out = np.zeros_like(w)
    out[order[:n]] = w[order[:n]]
    return out / out.sum()


def softmax(l, T):
    l = np.where(np.isnan(l), -np.inf, l.astype(np.float64))
    top = l.max()
    if top == -np.inf:
        return np.zeros_like(l)
    with np.errstate(invalid="ignore"):
        w = np.exp(np.where(l == top, 0.0, l - top) / T)
    w[w < 2.0 ** -45] = 0.0          # (weights are whole numbers of 2^-44)
    return w / w.sum()


def verify(parent, token, n, logits, draft, u, T=1.0, k=0, p=1.0, mp=0.0, Td=1.0):
    """(nodes, token, prob, tolerance of prob, near): ``near`` tells that a decision
    lies within what weights in units of 2^-44 leave open.  Each weight is off by
    2^-44 of the largest at most, so a partial sum of a distribution by e = V 2^-43
    of its largest probability; A times that for q's part of a residual, and a
    share of the residual by twice that over its sum."""
    row, nodes, near = 0, [], False
    Td = Td if Td > 0 else 1.0
    V = logits.shape[1]
    while True:
        kids = [i for i in range(n) if (i - 1 if parent is None else parent[i]) == row - 1 and i >= row]
        if not T > 0:
            l = np.where(np.isnan(logits[row]), -np.inf, logits[row].astype(np.float64))
            if l.max() == -np.inf:
                return nodes, -1, 0.0, 0.0, near
            t = int(np.argmax(l))
            nxt = next((i for i in kids if token[i] == t), None)
            if nxt is None:
                return nodes, t, 1.0, 0.0, near
            nodes.append(nxt)
            row = nxt + 1
            continue
        full = target(logits[row], T, k, p, mp)
        if full is None:
            return nodes, -1, 0.0, 0.0, near
        q0 = softmax(draft[row], Td) if kids and row < len(draft) else None
        P, q, N, Z, A, nxt, seen = full.copy(), None if q0 is None else q0.copy(), 1.0, 1.0, 0.0, None, set()
        for i in kids if q0 is not None else []:
            x = int(token[i])
            if not 0 <= x < V or x in seen or q0[x] <= 0:
                continue
            seen.add(x)
            e = V * 2.0 ** -43 * (full.max() + q0.max()) * (1 + A)
            # P and q are normalised here: times N and Z they are the parts of the whole
            left, right = u[i + 1] * q[x], P[x]
            near = near or abs(left - right) * N <= 4 * e * (1 + q0[x] / Z * (1 + N / Z))
            if left < right:
                nxt = i
                break
            rest = np.maximum(P - q, 0.0)
            A += N / Z
            N *= rest.sum()
            Z -= q0[x]
            q[x] = 0.0
            if N <= 1e-11:       # nothing is left of p; the library may see it differently
                near = near or N > 0
                P, N, A = full.copy(), 1.0, 0.0
                break
            P = rest / rest.sum()
            if q.sum() <= 1e-9:  # q's last token was tried
                near = near or len(seen) < (q0 > 0).sum()
                break
            q /= q.sum()
        if nxt is not None:
            nodes.append(nxt)
            row = nxt + 1
            continue
        cum = np.cumsum(P)
        mark = float(u[0]) * cum[-1]
        e = V * 2.0 ** -43 * (full.max() + (0.0 if q0 is None else q0.max())) * (1 + A) / N
        near = near or np.abs(cum[:-1] - mark).min(initial=1.0) <= 2 * e
        j = min(int((cum <= mark).sum()), int(np.flatnonzero(P > 0)[-1]))
        return nodes, j, float(P[j]), 2.0 ** -23 * float(P[j]) + 4 * e, near
