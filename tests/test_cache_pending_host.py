"""Refusals of the page operations' forms with pending tokens, without a GPU
(they return before any device call)."""
from __future__ import annotations

import pytest

from tests.test_cache_host import BAD_DESC, INVALID, UNSUPPORTED, A, desc, lib  # noqa: F401


def call(lib, name, c, **over):  # noqa: F811
    args = {"reserve_ex": dict(table=A, width=4, lens=A, want=A, R=2, pending=1, ok=A),
            "fork_ex": dict(table=A, width=4, lens=A, R=4, src=A, dst=A, n=2, pending=1, ok=A)}[name]
    assert set(over) <= set(args)
    args.update(over)
    return getattr(lib, "dartree_cache_" + name)(c, *args.values(), None)


REFUSED = [
    ("reserve_ex", dict(pending=-1), INVALID), ("reserve_ex", dict(want=None), INVALID), ("reserve_ex", dict(ok=None), INVALID),
    ("reserve_ex", dict(R=0), INVALID), ("reserve_ex", dict(R=4097), UNSUPPORTED),
    ("reserve_ex", dict(R=4096, width=1 << 20), UNSUPPORTED),
    ("fork_ex", dict(pending=-1), INVALID), ("fork_ex", dict(pending=-1, n=0), INVALID), ("fork_ex", dict(n=0), 0),
    ("fork_ex", dict(src=None), INVALID), ("fork_ex", dict(n=-1), INVALID), ("fork_ex", dict(n=1025), UNSUPPORTED),
    ("fork_ex", dict(n=1024, width=1 << 22), UNSUPPORTED),
]


@pytest.mark.parametrize("case", range(len(REFUSED)))
def test_refused_before_any_launch(lib, case):  # noqa: F811
    name, over, want = REFUSED[case]
    assert call(lib, name, desc(), **over) == want


@pytest.mark.parametrize("name", ["reserve_ex", "fork_ex"])
def test_bad_descriptors_are_refused(lib, name):  # noqa: F811
    for over in (*BAD_DESC, dict(refs=None)):
        assert call(lib, name, desc(**over)) == INVALID
