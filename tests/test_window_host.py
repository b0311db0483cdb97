"""Window attention, page plans and packed writes without a GPU: the refusals
of the C entry points (they return before any device call) and the workspace."""
from __future__ import annotations

import pytest

from speculative_decoding_draft_06_gb300 import build as cuda_build
from speculative_decoding_draft_06_gb300 import dartree as dtl
from tests.test_cache_host import A, BAD_DESC, INVALID, UNSUPPORTED, desc


@pytest.fixture(scope="module")
def lib():
    cuda_build.build()
    return dtl.load()


ARGS = {
    "window_attention": dict(layer=0, Q=A, qs=1024, q_rows=8, start=None, mask=None, n_nodes=None, table=A, width=4, lens=A,
                             R=2, B=3, max_len=100, offset=0, window=9, sinks=2, Hq=8, scale=0.1, zero=0, O=A, work=A,
                             work_bytes=1 << 40, err=None),
    "append_slots": dict(layer=0, K=A, V=A, ts=256, slot=A, n=4, err=None),
    "plan": dict(table=A, width=4, lens=A, count=A, R=2, offset=0, window=9, sinks=2, T=8, ok=A, start=A, row=A, pos=A,
                 slot=A, err=None),
}


def call(lib, name, c, **over):
    args = dict(ARGS[name])
    assert set(over) <= set(args)
    args.update(over)
    return getattr(lib, "dartree_cache_" + name)(c, *args.values(), None)


REFUSED = [
    ("window_attention", dict(Q=None), INVALID), ("window_attention", dict(O=None), INVALID),
    ("window_attention", dict(table=None), INVALID), ("window_attention", dict(lens=None), INVALID),
    ("window_attention", dict(Q=A + 8), INVALID), ("window_attention", dict(O=A + 2), INVALID),
    ("window_attention", dict(work=A + 4), INVALID), ("window_attention", dict(qs=1023), INVALID),
    ("window_attention", dict(qs=1016), INVALID), ("window_attention", dict(Hq=7), INVALID),
    ("window_attention", dict(Hq=0), INVALID), ("window_attention", dict(R=0), INVALID),
    ("window_attention", dict(B=-1), INVALID), ("window_attention", dict(max_len=-1), INVALID),
    ("window_attention", dict(window=-1), INVALID), ("window_attention", dict(sinks=-1), INVALID),
    ("window_attention", dict(scale=0.0), INVALID), ("window_attention", dict(scale=float("nan")), INVALID),
    ("window_attention", dict(layer=2), INVALID), ("window_attention", dict(q_rows=7), INVALID),
    ("window_attention", dict(q_rows=0, start=A), INVALID), ("window_attention", dict(start=A, n_nodes=A), INVALID),
    ("window_attention", dict(mask=A, B=1025, q_rows=3000), INVALID), ("window_attention", dict(width=0), INVALID),
    ("window_attention", dict(max_len=100000, R=1, window=0, B=0, work=None), INVALID),
    ("window_attention", dict(B=1 << 29, q_rows=1 << 31), UNSUPPORTED),
    ("window_attention", dict(R=65536, q_rows=1 << 31), UNSUPPORTED),
    ("window_attention", dict(max_len=(1 << 30) + 1), UNSUPPORTED),
    ("append_slots", dict(K=None), INVALID), ("append_slots", dict(V=None), INVALID), ("append_slots", dict(slot=None), INVALID),
    ("append_slots", dict(K=A + 2), INVALID), ("append_slots", dict(layer=2), INVALID), ("append_slots", dict(n=0), INVALID),
    ("append_slots", dict(ts=255), INVALID), ("append_slots", dict(ts=248), INVALID),
    ("plan", dict(table=None), INVALID), ("plan", dict(lens=None), INVALID), ("plan", dict(count=None), INVALID),
    ("plan", dict(ok=None), INVALID), ("plan", dict(start=None), INVALID), ("plan", dict(row=None), INVALID),
    ("plan", dict(pos=None), INVALID), ("plan", dict(slot=None), INVALID), ("plan", dict(R=0), INVALID),
    ("plan", dict(width=0), INVALID), ("plan", dict(T=-1), INVALID), ("plan", dict(window=-1), INVALID),
    ("plan", dict(sinks=-1), INVALID), ("plan", dict(R=4097), UNSUPPORTED), ("plan", dict(R=4096, width=1 << 19), UNSUPPORTED),
]


@pytest.mark.parametrize("name, over, status", REFUSED)
def test_refusals(lib, name, over, status):
    assert call(lib, name, desc(), **over) == status
    assert lib.dartree_last_error(None)


@pytest.mark.parametrize("bad", BAD_DESC)
@pytest.mark.parametrize("name", list(ARGS))
def test_bad_descriptors(lib, name, bad):
    assert call(lib, name, desc(**bad)) == INVALID


def test_plan_needs_holders_and_slots_of_31_bits(lib):
    assert call(lib, "plan", desc(refs=None)) == INVALID
    assert call(lib, "plan", desc(pages=1 << 25, page_tokens=64)) == UNSUPPORTED


def test_workspace(lib):
    work = lib.dartree_cache_window_attention_workspace
    # sizes outside the call's limits have none, as calls that need no joining
    for bad in ((0, 0, 100, 9, 0, 1, 8, 2, 128), (1, -1, 100, 9, 0, 1, 8, 2, 128), (1, 1025, 100, 9, 0, 0, 8, 2, 128),
                (1, 0, -1, 9, 0, 1, 8, 2, 128), (1, 0, 100, 9, -1, 1, 8, 2, 128), (1, 0, 100, 9, 0, 1, 7, 2, 128),
                (1, 0, 100, 9, 0, 1, 8, 2, 96), (1, 1 << 29, 100, 9, 0, 1, 8, 2, 128), (1, 0, 100, 9, 0, 1, 8, 2, 128)):
        assert work(*bad) == 0
    # a window bounds the keys and so the splits
    far = work(1, 0, 1 << 20, 0, 0, 1, 32, 8, 128)
    assert far == lib.dartree_cache_attention_workspace(1, 0, 1 << 20, 32, 8, 128) > 0
    assert work(1, 0, 1 << 20, 1 << 30, 0, 1, 32, 8, 128) == far
    assert work(1, 0, 1 << 20, 100, 4, 1, 32, 8, 128) < far


VERIFY = dict(parent=A, token=A, n_out=A, logits=A, bf16=0, rs=4000, ws=1000, draft=A, dbf16=1, drs=3000, dws=1000, rows=3, V=1000,
              R=2, B=3, T=A, k=A, p=A, m=A, Td=A, u=A, max_len=4, len=A, nodes=A, bonus=A, prob=A)


@pytest.mark.parametrize("over, status", [
    (dict(token=None), INVALID), (dict(n_out=None), INVALID), (dict(logits=None), INVALID), (dict(draft=None), INVALID),
    (dict(u=None), INVALID), (dict(len=None), INVALID), (dict(nodes=None), INVALID), (dict(bonus=None), INVALID),
    (dict(prob=None), INVALID), (dict(V=0), INVALID), (dict(R=0), INVALID), (dict(B=0), INVALID), (dict(rows=0), INVALID),
    (dict(max_len=0), INVALID), (dict(ws=999), INVALID), (dict(dws=999), INVALID), (dict(rs=-1), INVALID),
    (dict(drs=-1), INVALID), (dict(logits=A + 2), INVALID), (dict(draft=A + 1), INVALID),
    (dict(V=(1 << 18) + 1, ws=1 << 19, dws=1 << 19), UNSUPPORTED), (dict(B=1025), UNSUPPORTED),
    (dict(R=(1 << 24) + 1), UNSUPPORTED)])
def test_verify_refusals(lib, over, status):
    assert lib.dartree_verify(*{**VERIFY, **over}.values(), None) == status
    assert lib.dartree_last_error(None)


def test_verification_reference():
    """The reference's own arithmetic on a case by hand: p = (1/2, 1/2, 0), q = (1/4, 0, 3/4)."""
    import numpy as np

    from tests import verify_ref as ref
    with np.errstate(divide="ignore"):
        z, d = np.log([[0.5, 0.5, 0.0]] * 3), np.log([[0.25, 0.0, 0.75]] * 3)
    par = [-1, -1]
    # token 2: p = 0, never accepted; then max(p - q, 0) = (1/4, 1/2, 0): token 0 is left of q, with
    # certainty, and accepted with probability 1/3
    for u, nodes in ((0.33, [1]), (0.34, [])):
        got = ref.verify(par, [2, 0], 2, z, d, [0.5, 0.0, u])
        assert got[0] == nodes
    # rejected as well: max((1/3, 2/3, 0) - (1, 0, 0), 0): token 1
    assert got[1] == 1 and abs(got[2] - 1.0) < 1e-12
    # token 0 first: accepted (p > q)
    assert ref.verify(par, [0, 2], 2, z, d, [0.5, 0.99, 0.0])[0] == [0]
