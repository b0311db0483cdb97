"""The paged 4-bit cache and sampling without a GPU: the refusals of the C
entry points (they return before any device call), the format's sizes, the
workspace, and the reference arithmetic that the GPU tests compare with."""
from __future__ import annotations

import ctypes

import numpy as np
import pytest

from speculative_decoding_draft_06_gb300 import build as cuda_build
from speculative_decoding_draft_06_gb300 import dartree as dtl
from tests import cache_ref as ref

INVALID, UNSUPPORTED = 1, 2
A = 0x10000000  # an address that is never dereferenced


@pytest.fixture(scope="module")
def lib():
    cuda_build.build()
    return dtl.load()


def desc(**over):
    d = dict(pool=A, refs=A, layers=2, pages=10, page_tokens=64, Hkv=2, dh=128, k_scale=1.0, v_scale=1.0)
    d.update(over)
    return ctypes.byref(dtl.Cache(*(d[n] for n, _ in dtl.Cache._fields_)))


BAD_DESC = [dict(Hkv=65536), dict(pool=None), dict(pool=A + 8), dict(layers=0), dict(pages=0), dict(Hkv=0), dict(page_tokens=48),
            dict(page_tokens=256), dict(dh=96), dict(dh=256), dict(k_scale=3.0), dict(v_scale=0.0),
            dict(v_scale=-1.0), dict(k_scale=2.0 ** 65), dict(k_scale=float("nan")), dict(v_scale=float("inf"))]


def call(lib, name, c, **over):
    args = {
        "append": dict(layer=0, K=A, V=A, rs=256 * 4, ts=256, table=A, width=4, lens=A, offset=0, count=None, R=2,
                       n=4, err=None),
        "read": dict(layer=0, K=A, V=A, table=A, width=4, lens=A, offset=0, count=None, R=2, n=4, err=None),
        "attention": dict(layer=0, Q=A, qs=1024, mask=A, n_nodes=None, table=A, width=4, lens=A, R=2, B=3,
                          max_len=100, Hq=8, scale=0.1, O=A, work=A, work_bytes=1 << 40, err=None),
        "reserve": dict(table=A, width=4, lens=A, want=A, R=2, ok=A),
        "fork": dict(table=A, width=4, lens=A, R=4, src=A, dst=A, n=2, ok=A),
        "commit": dict(table=A, width=4, lens=A, nodes=A, len=A, R=2, max_len=4, extra=1, err=None),
        "release": dict(table=A, width=4, lens=A, R=2, rows=A, keep=A, n=2, err=None),
        "copy_pages": dict(src=A, dst=A, n=2, err=None),
    }[name]
    assert set(over) <= set(args)
    args.update(over)
    return getattr(lib, "dartree_cache_" + name)(c, *args.values(), None)


REFUSED = [
    ("append", dict(K=None), INVALID), ("append", dict(V=None), INVALID), ("append", dict(K=A + 2), INVALID),
    ("append", dict(table=None), INVALID), ("append", dict(lens=None), INVALID), ("append", dict(layer=2), INVALID),
    ("append", dict(layer=-1), INVALID), ("append", dict(R=0), INVALID), ("append", dict(n=0), INVALID),
    ("append", dict(width=0), INVALID), ("append", dict(ts=255), INVALID), ("append", dict(ts=128), INVALID),
    ("append", dict(rs=4), INVALID), ("append", dict(rs=-1024), INVALID),
    ("append", dict(R=1 << 30, n=1 << 30), UNSUPPORTED),
    ("read", dict(K=None), INVALID), ("read", dict(V=A + 8), INVALID), ("read", dict(layer=5), INVALID),
    ("read", dict(n=-1), INVALID), ("read", dict(table=None), INVALID),
    ("attention", dict(Q=None), INVALID), ("attention", dict(O=None), INVALID), ("attention", dict(O=A + 2), INVALID),
    ("attention", dict(mask=None), INVALID), ("attention", dict(table=None), INVALID),
    ("attention", dict(lens=None), INVALID), ("attention", dict(B=-1), INVALID), ("attention", dict(B=1025), INVALID),
    ("attention", dict(Hq=7), INVALID), ("attention", dict(Hq=0), INVALID), ("attention", dict(scale=0.0), INVALID),
    ("attention", dict(scale=float("nan")), INVALID), ("attention", dict(scale=float("inf")), INVALID),
    ("attention", dict(qs=1023), INVALID), ("attention", dict(qs=512), INVALID), ("attention", dict(R=0), INVALID),
    ("attention", dict(max_len=-1), INVALID), ("attention", dict(layer=2), INVALID),
    ("attention", dict(max_len=100000, work=None), INVALID),
    ("attention", dict(max_len=100000, work_bytes=100), INVALID),
    ("attention", dict(R=70000), UNSUPPORTED), ("attention", dict(scale=-0.1), INVALID),
    ("commit", dict(R=(1 << 24) + 1), UNSUPPORTED), ("commit", dict(max_len=1 << 30), UNSUPPORTED),
    ("reserve", dict(want=None), INVALID), ("reserve", dict(ok=None), INVALID), ("reserve", dict(R=0), INVALID),
    ("reserve", dict(R=4097), UNSUPPORTED), ("reserve", dict(R=4096, width=1 << 20), UNSUPPORTED),
    ("fork", dict(src=None), INVALID), ("fork", dict(n=-1), INVALID), ("fork", dict(n=1025), UNSUPPORTED),
    ("fork", dict(ok=None), INVALID), ("fork", dict(n=0), 0),
    ("commit", dict(nodes=None), INVALID), ("commit", dict(len=None), INVALID), ("commit", dict(max_len=0), INVALID),
    ("commit", dict(extra=-1), INVALID), ("commit", dict(lens=None), INVALID),
    ("release", dict(rows=None), INVALID), ("release", dict(n=-1), INVALID), ("release", dict(n=0), 0),
    ("copy_pages", dict(src=None), INVALID), ("copy_pages", dict(n=-1), INVALID),
    ("copy_pages", dict(n=65536), UNSUPPORTED), ("copy_pages", dict(n=0), 0),
]


@pytest.mark.parametrize("case", range(len(REFUSED)))
def test_refused_before_any_launch(lib, case):
    name, over, want = REFUSED[case]
    assert call(lib, name, desc(), **over) == want
    if want:
        assert lib.dartree_last_error(None)


@pytest.mark.parametrize("case", range(len(BAD_DESC)))
@pytest.mark.parametrize("name", ["append", "read", "attention", "reserve", "fork", "commit", "release", "copy_pages"])
def test_bad_descriptors_are_refused(lib, name, case):
    assert call(lib, name, desc(**BAD_DESC[case])) == INVALID


@pytest.mark.parametrize("name", ["reserve", "fork", "release"])
def test_the_allocator_needs_refs(lib, name):
    assert call(lib, name, desc(refs=None)) == INVALID


def test_a_scale_that_overflows_with_the_keys_unit_is_refused(lib):
    assert call(lib, "attention", desc(k_scale=2.0 ** 64), scale=1e20) == INVALID
    assert call(lib, "attention", desc(k_scale=2.0 ** -64), scale=3.1e38) == INVALID


def test_page_bytes(lib):
    assert lib.dartree_cache_page_bytes(64, 8, 128) == 64 * 8 * 144
    assert lib.dartree_cache_page_bytes(16, 1, 64) == 16 * 72
    for P, Hkv, dh in ((8, 1, 64), (64, 0, 64), (64, 1, 32), (65, 1, 64)):
        assert lib.dartree_cache_page_bytes(P, Hkv, dh) == 0


def test_workspace(lib):
    need = lib.dartree_cache_attention_workspace
    assert need(1, 0, 0, 8, 8, 128) == 0            # no keys: one share
    assert need(1, 0, 100000, 8, 8, 128) > 0        # a long sequence is shared out
    for bad in ((0, 0, 10, 8, 8, 128), (1, -1, 10, 8, 8, 128), (1, 0, -1, 8, 8, 128), (1, 0, 10, 8, 3, 128),
                (1, 0, 10, 8, 0, 128), (1, 0, 10, 8, 8, 96)):
        assert need(*bad) == 0


def test_sample_refusals(lib):
    ok = dict(logits=A, bf16=0, stride=100, V=100, rows=4, per=2, T=None, k=None, p=None, m=None, u=A, token=A, prob=A)
    for over, want in ((dict(logits=None), INVALID), (dict(u=None), INVALID), (dict(token=None), INVALID),
                       (dict(prob=None), INVALID), (dict(V=0), INVALID), (dict(rows=0), INVALID),
                       (dict(per=0), INVALID), (dict(stride=99), INVALID),
                       (dict(V=(1 << 18) + 1, stride=1 << 20), UNSUPPORTED)):
        assert lib.dartree_sample(*dict(ok, **over).values(), None) == want


def test_reference_quantisation():
    """The reference's grids are the formats' values and its rounding is to
    nearest, ties to even."""
    assert ref.E4M3[-1] == 448.0 and ref.E4M3[1] == 2.0 ** -9 and len(ref.E4M3) == 127
    x = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0, 9.0, 0.2, 0.3, 2.4])
    assert list(ref.E2M1[ref.nearest(x, ref.E2M1)]) == [0, 1, 1, 2, 2, 4, 4, 6, 6, 0, 0.5, 2]
    g = np.random.default_rng(0)
    y = g.standard_normal((5, 64)) * 10.0 ** g.integers(-2, 3, (5, 64))
    c, s = ref.quantise(y)
    v = ref.values(c, s)
    # a scale is within 2^-4 of max/6, so a value is within half a step (1 of 6) of a block's range,
    # with the largest clipped by at most the scale's rounding
    top = np.abs(y.reshape(5, 4, 16)).max(-1, keepdims=True)
    assert (np.abs(v - y).reshape(5, 4, 16) <= top / 6 * (1 + 2.0 ** -4)).all()


def test_reference_sampling():
    l = np.log(np.array([0.1, 0.4, 0.2, 0.3]))
    assert [ref.sample_row(l, 1.0, 0, 1.0, 0.0, u)[0] for u in (0.05, 0.2, 0.6, 0.9)] == [0, 1, 2, 3]
    assert [ref.sample_row(l, 1.0, 2, 1.0, 0.0, u)[0] for u in (0.1, 0.6)] == [1, 3]
    assert [ref.sample_row(l, 1.0, 0, 0.65, 0.0, u)[0] for u in (0.1, 0.6)] == [1, 3]
    assert ref.sample_row(l, 1.0, 0, 1.0, 0.8, 0.9)[0] == 1
    assert ref.sample_row(l, 0.0, 0, 1.0, 0.0, 0.9)[:2] == (1, 1.0)
    assert ref.sample_row(np.full(4, -np.inf), 1.0, 0, 1.0, 0.0, 0.5)[:2] == (-1, 0.0)
