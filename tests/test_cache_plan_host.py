"""How a call of the attention over the cache is cut, as far as its workspace
shows it (no GPU)."""
from __future__ import annotations

import pytest

from tests.test_cache_host import lib  # noqa: F401

SMS, PER_SM, DH = 152, 3, 128


@pytest.mark.parametrize("R,Hkv,keys,splits,workspace", [
    (1, 8, 1000, 4, False),       # 32 CTAs: clusters
    (4, 8, 8000, 11, True),       # more splits than a cluster has CTAs
    (8, 8, 4100, 6, False), (8, 8, 6000, 8, True),   # 384 CTAs; 512 are not resident at once
    (6, 8, 1000, 4, False),
    (16, 8, 4100, 4, True), (32, 8, 1000, 2, True), (19, 8, 1000, 3, False),
    (64, 8, 2000, 1, False), (64, 8, 16001, 8, True), (128, 8, 2500, 2, True)])
def test_splits_join_in_clusters_where_all_are_resident(lib, R, Hkv, keys, splits, workspace):  # noqa: F811
    got = lib.dartree_cache_attention_workspace(R, 0, keys, 4 * Hkv, Hkv, DH)
    assert got == (R * Hkv * splits * 8 * (DH + 4) * 4 if workspace else 0)
    assert workspace == (splits > 8 or (splits > 1 and R * Hkv * splits > SMS * PER_SM))
