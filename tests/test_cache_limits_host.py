"""Sizes at the ends of what 32 bits hold: refused before any device call."""
from __future__ import annotations

import pytest

from tests.test_cache_host import UNSUPPORTED, call, desc, lib  # noqa: F401
from tests.test_window_host import call as window_call

MOST = 2 ** 31 - 1


@pytest.mark.parametrize("n", [MOST, MOST - 1, MOST - 2, MOST - 6, MOST - 7])
@pytest.mark.parametrize("dh", [64, 128])
def test_tokens_of_one_write(lib, n, dh):  # noqa: F811
    """More tokens than a launch has warps for."""
    c = dict(Hkv=64, dh=dh)
    assert window_call(lib, "append_slots", desc(**c), n=n, ts=64 * dh) == UNSUPPORTED
    assert call(lib, "append", desc(**c), R=1, n=n, ts=64 * dh) == UNSUPPORTED
    assert call(lib, "read", desc(**c), R=1, n=n) == UNSUPPORTED
