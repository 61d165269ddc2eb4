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


def test_step_takes_any_form_of_a_phase(lk):
    # tuples of cells, as append and decode take them, and the current tokens where a cell shares
    from loop_aware_quantized_b200 import steps

    class Cache:
        shared, newest, calls = np.array([True, False, False, False]), "newest", []

        def grow(self, ones, slots, stream=None):
            self.calls.append(("grow", ones))

        def append(self, cells, k, v, slots, stream=None):
            self.calls.append(("append", list(cells), k, slots))

        def decode(self, cells, q, cur_k=None, cur_v=None, out=None, lse=None, stream=None):
            self.calls.append(("decode", list(cells), cur_k))

    for forms in (((0, 1), (2, 3)), ([0, 1], [2, 3]), (range(2), range(2, 4)), (np.arange(2), np.arange(2, 4))):
        cache = Cache()
        cache.calls = []
        steps.paged_decode_step(cache, forms, "ones", "slots", "qq", "kK", "vV", ["o", "p"])
        assert cache.calls == [("grow", "ones"), ("append", [0, 1], "k", "newest"), ("decode", [0, 1], "k"),
                               ("append", [2, 3], "K", "newest"), ("decode", [2, 3], None)]


def test_shared_is_a_list_of_cells_not_a_mask(lk):
    # (as an index, a truth value would mark every cell or none)
    from loop_aware_quantized_b200 import PagedCache
    make = lambda shared: PagedCache(2, 2, 1, 64, 4, 16, 2, 4, shared=shared, device="cpu")  # noqa: E731
    for shared in (np.array([True, False, False, False]), [False, True], [True], [0.5], np.array([1 << 32]), ["x"]):
        with pytest.raises(lk.LoopKVError) as e:
            make(shared)
        assert e.value.status == 1
    for shared in ([1], (1,), range(1, 2), np.array([1]), {1}, np.array([1.0]), iter([1])):
        assert make(shared).shared.tolist() == [False, True, False, False]
    assert not make(()).shared.any() and not make(np.array([], np.int32)).shared.any()
