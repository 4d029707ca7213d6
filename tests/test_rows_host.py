"""The shared-prefix, weighing, eviction and cross-attention calls refuse bad
arguments on the host, and the oracle's eviction order is what it says."""
import ctypes

import numpy as np
import pytest

from oracle import rows as R


@pytest.fixture(scope="module")
def N():
    from conftest import build_library
    build_library()
    from dynamic_sparse_kv_gb300 import _native
    return _native


def test_null_arguments_are_refused(N):
    L = N.lib
    kv = N.fastocr_kv(None, None, None, None, 1)
    g = N.fastocr_groups(None, None, 1, 0)
    w = N.fastocr_weights(None, None, None, None, None, 1)
    b = ctypes.byref
    assert L.fastocr_shared_attend(None, None, b(kv), b(g), None, None, None, 0, None) == N.FASTOCR_ERR_NULL
    assert L.fastocr_weigh_attend(None, None, b(kv), b(w), None, None) == N.FASTOCR_ERR_NULL
    assert L.fastocr_evict(None, b(kv), b(w), 1, 0, None, None) == N.FASTOCR_ERR_NULL
    assert L.fastocr_cross_attend(None, None, b(kv), None, 1, None, None, 0, None) == N.FASTOCR_ERR_NULL
    assert L.fastocr_rows_workspace(None, 1) == N.FASTOCR_ERR_NULL
    with pytest.raises(N.FastOCRError):
        N.fastocr_rows_workspace(None, 1)


def test_evict_order_of_the_oracle():
    pos = [9, 8, 7, 6, 5]
    stay, moves = R.evict_moves([1, 5, 5, 2, 7], pos, 5, seen=10, budget=2, recent=0)
    assert stay == [1, 4] and moves == [(4, 0)]
    stay, _ = R.evict_moves([1, 5, 5, 2, 7], pos, 5, seen=10, budget=2, recent=1)
    assert stay == [0, 4]                       # position 9 is recent
    stay, moves = R.evict_moves([0, 5, 5, 5, 0], pos, 5, seen=10, budget=2, recent=0)
    assert stay == [1, 2] and moves == [(2, 0)]  # ties to the lower row
    stay, _ = R.evict_moves([np.nan, -1, -np.inf, np.inf, 0], pos, 5, seen=10, budget=4, recent=0)
    assert stay == [1, 2, 3, 4]
    stay, moves = R.evict_moves([3, 2, 1], pos, 3, seen=10, budget=3, recent=0)
    assert stay == [0, 1, 2] and moves == []


def test_weights_of_the_oracle():
    p = np.array([[0.25, 0.5, 0.25], [0.0, 0.5, 0.5]])     # two heads of one KV head
    mass, pos = R.add_weights([[9.0, 9.0]], [[1, 1]], p, 3, 1, 30, 1)
    assert mass.tolist() == [[10.0, 0.75]] and pos.tolist() == [[1, 29]]
