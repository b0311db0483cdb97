"""Rows whose last tokens are counted before they are written (commit's bonus
token): fork and reserve give each row pages of its own for them."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from speculative_decoding_draft_06_gb300 import dartree as dtl
from tests import cache_ref as ref
from tests.test_gpu_cache import cu, host, same, sequences

pytestmark = pytest.mark.gpu


class Pages(ref.Pages):
    """The page operations with pending tokens, one row and page at a time."""

    def reserve(self, want, pending=0):
        R, width = self.table.shape
        ok, out = np.zeros(R, np.int32), False
        lens, want = [int(x) for x in self.lens], [int(x) for x in want]
        need = [-(-(n + w) // self.P) for n, w in zip(lens, want)]
        refused = [lens[r] < 0 or want[r] < 0 or need[r] > width or
                   (want[r] + pending > 0 and any(self.refs[self.table[r, s]] > 1 for s in range(
                       max(lens[r] - pending, 0) // self.P, min(self.held(r), need[r])))) for r in range(R)]
        for r in range(R):
            if refused[r]:
                continue
            lack = max(0, need[r] - self.held(r))
            free = np.flatnonzero(self.refs == 0)
            out = out or lack > len(free)
            if lack and out:
                continue
            ok[r] = 1
            for page in free[:lack]:
                self.table[r, self.held(r)] = page
                self.refs[page] = 1
        return ok

    def fork(self, src, dst, pending=0):
        R, width = self.table.shape
        ok, out = np.zeros(len(src), np.int32), False
        empty = [0 <= d < R and self.held(d) == 0 for d in dst]
        for i, (s, d) in enumerate(zip(src, dst)):
            if not (0 <= s < R and 0 <= d < R) or d in src or d in dst[:i] or not empty[i]:
                continue
            n = int(self.lens[s])
            done = max(n - pending, 0)
            need, whole = -(-n // self.P), done // self.P
            if n < 0 or need > width or -(-done // self.P) > self.held(s):
                continue
            free = np.flatnonzero(self.refs == 0)
            out = out or need - whole > len(free)
            if need > whole and out:
                continue
            ok[i] = 1
            for j in range(whole):
                self.table[d, j] = self.table[s, j]
                self.refs[self.table[s, j]] += 1
            for j in range(whole, need):
                page = int(free[j - whole])
                self.refs[page] = 1
                self.table[d, j] = page
                if j == whole and done % self.P:
                    self.pool[:, page] = self.pool[:, self.table[s, whole]]
            self.lens[d] = n
        return ok


@pytest.mark.parametrize("behind", [0, 1, 2])
def test_rows_forked_behind_a_commit_write_their_own_bonus_tokens(behind):
    """commit(extra=1) leaves a row at a page's end (or one or two tokens
    behind it); the rows forked there append different bonus tokens at offset
    -1, and each reads its own."""
    P, Hkv, dh = 16, 2, 64
    g = np.random.default_rng(behind)
    bf = lambda *s: torch.from_numpy(g.standard_normal(s)).to(torch.bfloat16).cuda()  # noqa: E731
    cache = dtl.KVCache(2, 20, page_tokens=P, Hkv=Hkv, dh=dh)
    table, lens = cu(np.full((3, 6), -1)), cu([0, 0, 0])
    start = 44 + behind
    assert host(cache.reserve(table, lens, cu([start + 10, 0, 0]))).tolist() == [1, 1, 1]
    K = bf(3, start + 8, Hkv, dh)
    for layer in range(2):
        cache.append(layer, K, K, table, lens, count=cu([start + 8, 0, 0]))
    lens[0] = start
    cache.commit(table, lens, cu([[0, 2, 5], [-1] * 3, [-1] * 3]), cu([3, 0, 0]), extra=1)
    lens[1:] = 0
    assert host(lens).tolist() == [start + 4, 0, 0]           # the token at start + 3 is not written
    cache.release(table, lens, cu([0]), lens[:1].clone())
    assert host(cache.fork(table, lens, cu([0, 0]), cu([1, 2]), pending=1)).tolist() == [1, 1]
    t = host(table)
    at = (start + 3) // P
    assert (t[:, :at] == t[0, :at]).all() and len(set(t[:, at])) == 3 and (t[:, at] >= 0).all()
    assert host(cache.reserve(table, lens, cu([4, 0, 9]), pending=1)).tolist() == [1, 1, 1]
    own = bf(3, 1, Hkv, dh)
    for layer in range(2):
        cache.append(layer, own, -own, table, lens, offset=-1)
    before = K[0, [*range(start), start, start + 2, start + 5]]
    for layer in range(2):
        k, v = cache.read(layer, table, cu([0, 0, 0]), start + 4)
        for r in range(3):
            q = lambda x: ref.values(*ref.quantise(host(x.double())))  # noqa: E731
            assert np.array_equal(host(k[r].double()), q(torch.cat([before, own[r]])))
            assert np.array_equal(host(v[r].double()), q(torch.cat([before, -own[r]])))
    cache.check()


def test_a_row_whose_pending_token_lies_in_a_shared_page_is_refused():
    """Forked without its pending token: reserve says so before anything is
    written, and a fork that knows of it has a page of its own."""
    cache = dtl.KVCache(1, 12, page_tokens=16, Hkv=1, dh=64)
    table, lens = cu(np.full((3, 4), -1)), cu([0, 0, 0])
    assert host(cache.reserve(table, lens, cu([32, 0, 0]))).tolist() == [1, 1, 1]
    lens[0] = 32
    assert host(cache.fork(table, lens, cu([0]), cu([1]))).tolist() == [1]
    before = host(table)
    assert host(cache.reserve(table, lens, cu([3, 0, 5]), pending=1)).tolist() == [0, 0, 1]
    t = host(table)
    assert (t[:2] == before[:2]).all() and t[2, 0] >= 0 and (t[2, 1:] == -1).all()
    cache.release(table, lens, cu([2]), cu([0]))
    assert host(cache.fork(table, lens, cu([1]), cu([2]), pending=1)).tolist() == [1]
    assert host(cache.reserve(table, lens, cu([0, 0, 5]), pending=1)).tolist() == [0, 0, 1]
    cache.release(table, lens, cu([1]), cu([0]))
    assert host(cache.reserve(table, lens, cu([3, 0, 0]), pending=1)).tolist() == [1, 1, 1]
    # a length lowered by hand to a page's end: the page behind it is shared
    lens.copy_(cu([16, 0, 33]))
    cache.release(table, lens, cu([0, 2]), cu([0, 0]))
    assert host(cache.reserve(table, lens, cu([48, 0, 0]))).tolist() == [1, 1, 1]
    lens[0] = 48
    assert host(cache.fork(table, lens, cu([0]), cu([1]))).tolist() == [1]
    lens[0] = 16
    assert host(cache.reserve(table, lens, cu([1, 1, 0]))).tolist() == [0, 1, 1]
    cache.check()


@pytest.mark.parametrize("seed", range(12))
def test_fork_and_reserve_with_pending_tokens(seed):
    """Against the model: any number of pending tokens, from none to more than
    the row has; too few pages; sources that have no page for them."""
    g = np.random.default_rng(500 + seed)
    P, dh, Hkv = int(g.choice([16, 32, 64, 128])), int(g.choice([64, 128])), int(g.integers(1, 4))
    R, S, width = 7, 10, 6
    cache, want, table, lens = sequences(g, R, P, Hkv, dh, 3, width, 90, S)
    want = Pages(want.pool, want.refs, want.table, want.lens, P)
    pending = [0, 1, 1, 2, P - 1, P, P + 1, 40, 3 * P, 10 ** 6, 2 ** 31 - 1, 1][seed]
    if seed in (1, 2, 11):                 # lengths around the pages' ends, some without a page for the last token
        for r in range(R):
            h = want.held(r)
            want.lens[r] = max(0, h * P + int(g.integers(-1, 2))) if h else 0
        lens.copy_(cu(want.lens))
    if seed % 3 == 2:                      # few pages
        busy = g.permutation(np.flatnonzero(want.refs == 0))
        want.refs[busy[int(g.integers(1, 9)):]] = 1
        cache.refs.copy_(cu(want.refs))
    src, dst = g.integers(0, R, S), R + g.permutation(S)
    if seed >= 8:
        src[0], dst[1], dst[2] = -1, R + S, 0
    ok = cache.fork(table, lens, cu(src), cu(dst), pending=pending)
    assert np.array_equal(host(ok), want.fork(list(src), list(dst), pending))
    same(cache, want, table, lens)
    for _ in range(2):
        w = g.integers(0, 2 * P, R + S)
        w[g.random(R + S) < 0.4] = 0
        ok = cache.reserve(table, lens, cu(w), pending=pending)
        assert np.array_equal(host(ok), want.reserve(w, pending))
        same(cache, want, table, lens)
        pending = 0
    cache.check()


def test_a_shared_page_is_not_written():
    """append leaves a page that two rows hold as it is and flags the token;
    tokens of the row's own pages are written."""
    P, Hkv, dh = 16, 3, 128
    cache = dtl.KVCache(1, 8, page_tokens=P, Hkv=Hkv, dh=dh)
    table, lens = cu(np.full((2, 4), -1)), cu([0, 0])
    assert host(cache.reserve(table, lens, cu([32, 0]))).tolist() == [1, 1]
    K = torch.randn(2, 20, Hkv, dh, device="cuda").to(torch.bfloat16)
    cache.append(0, K, K, table, lens, count=cu([20, 0]))
    lens[0] = 32
    assert host(cache.fork(table, lens, cu([0]), cu([1]))).tolist() == [1]
    assert host(cache.reserve(table, lens, cu([20, 20]))).tolist() == [1, 1]
    cache.check()
    pool = cache.pool.clone()
    cache.append(0, -K, -K, table, lens, offset=-4)          # positions 28 .. 47: 28 .. 31 are shared
    with pytest.raises(dtl.DartreeError):
        cache.check()
    t = host(table)
    assert torch.equal(cache.pool[0, t[0, :2]], pool[0, t[0, :2]])
    k, _ = cache.read(0, table, lens, 16)
    assert np.array_equal(host(k.double()), -ref.values(*ref.quantise(host(K[:, 4:].double()))))
    cache.append(0, -K, -K, table, lens)                     # their own pages alone
    cache.check()
    cache.release(table, lens, cu([1]), cu([0]))
    cache.append(0, -K, -K, table, lens, offset=-4, count=cu([20, 0]))
    cache.check()
    k, _ = cache.read(0, table, lens, 20, offset=-4)
    assert np.array_equal(host(k[0].double()), -ref.values(*ref.quantise(host(K[0].double()))))
