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


@pytest.mark.parametrize("B, Hq", [(1023, 1 << 30), (1024, MOST), (1023, MOST), (1, 1 << 30)])
def test_rows_of_one_head(lib, B, Hq):  # noqa: F811
    """More than 2^30 rows per key/value head."""
    assert lib.dartree_cache_attention_workspace(1, B, 100, Hq, 1, 64) == 0
    c = dict(Hkv=1, dh=64)
    assert call(lib, "attention", desc(**c), R=1, B=B, Hq=Hq, qs=64 * Hq) == UNSUPPORTED
    assert window_call(lib, "window_attention", desc(**c), R=1, B=B, Hq=Hq, qs=64 * Hq, q_rows=B + 1) == UNSUPPORTED
