"""Paged cells without a GPU: lists of cells that are no cells, and the step's
forms of a phase."""

import numpy as np
import pytest


@pytest.fixture(scope="module")
def lk():
    from loop_aware_quantized_b200 import build
    build.build()
    from loop_aware_quantized_b200 import loopkv
    return loopkv


def test_cells_that_32_bits_lose_are_refused(lk):
    # 2^32 is not cell 0, and half a cell is none
    from loop_aware_quantized_b200 import PagedCache
    cache = PagedCache(2, 2, 1, 64, 4, 16, 2, 4, device="cpu")
    for cells in (np.array([1 << 32]), np.array([0.5]), [0, 1.5], np.array([-(1 << 32)]), np.array([np.nan]),
                  [1 << 40], ["x"], [None], np.array([(1 << 32) + 1], np.uint64)):
        for call in (lambda: cache.append(cells, None, None, None), lambda: cache.decode(cells, None)):
            with pytest.raises(lk.LoopKVError, match="cells") as e:
                call()
            assert e.value.status == 1
    for cells in (range(2), (0, 1), [np.int64(1)], np.array([0.0, 1.0]), np.array([[0, 1]], np.uint8)):
        with pytest.raises(lk.LoopKVError, match="k_pages must"):    # the next argument's turn
            cache.append(cells, None, None, None)
