"""Paged cells without a GPU: the C entry points and the binding refuse what
they cannot do before any CUDA call, and the 64-bit forms the GPU tests compare
with say what the definitions say."""

import ctypes

import numpy as np
import pytest

from tests import paged_reference as R


@pytest.fixture(scope="module")
def lk():
    from loop_aware_quantized_b200 import build
    build.build()
    from loop_aware_quantized_b200 import loopkv
    return loopkv


FAKE = ctypes.c_void_p(1 << 20)      # aligned, never dereferenced on these paths
ODD = ctypes.c_void_p((1 << 20) + 2)
INVALID = 1


def _map(lk, batch=2, page_size=16, max_pages=4, n_pages=8, n_rows=2, ptrs=None, slots=FAKE,
         newest=None, status=None):
    p = [FAKE] * 8 if ptrs is None else ptrs      # len new table free count | starts | len_out count_out
    return lk.loopkv_page_map(batch, page_size, max_pages, n_pages, n_rows, *p[:5], slots, p[5],
                              newest, *p[6:], status, None)


def _release(lk, batch=2, page_size=16, max_pages=4, n_pages=8, ptrs=None, status=None):
    p = [FAKE] * 7 if ptrs is None else ptrs
    return lk.loopkv_page_release(batch, page_size, max_pages, n_pages, *p, status, None)


@pytest.mark.parametrize("kw", [
    dict(batch=0), dict(batch=-1), dict(batch=4097), dict(page_size=0), dict(page_size=1025),
    dict(max_pages=0), dict(max_pages=(1 << 18) + 1), dict(n_pages=0), dict(n_pages=1 << 27),
    dict(status=ODD)])
def test_page_calls_refuse_sizes(lk, kw):
    assert _map(lk, **kw) == INVALID
    assert _release(lk, **kw) == INVALID


def test_page_calls_refuse_pointers(lk):
    for i in range(8):
        for bad in (None, ODD):
            assert _map(lk, ptrs=[bad if j == i else FAKE for j in range(8)]) == INVALID
    for i in range(7):
        for bad in (None, ODD):
            assert _release(lk, ptrs=[bad if j == i else FAKE for j in range(7)]) == INVALID
    assert _map(lk, newest=ODD) == INVALID
    assert _map(lk, slots=ODD) == INVALID
    assert _map(lk, n_rows=-1) == INVALID
    assert _map(lk, n_rows=(1 << 30) + 1) == INVALID


def _pool(lk, n_cells=2, n_pages=4, page_size=16, heads=2, dim=64, fmt=0, k=1 << 20, v=1 << 20,
          meta=None):
    return lk.loopkv_page_pool(n_cells, n_pages, page_size, heads, dim, fmt, k, v, meta)


BAD_POOLS = [dict(n_cells=0), dict(n_pages=0), dict(page_size=0), dict(page_size=1025),
             dict(heads=0), dict(heads=65537), dict(dim=96), dict(fmt=3), dict(fmt=-1),
             dict(k=None), dict(v=None), dict(k=(1 << 20) + 8), dict(meta=1 << 20), dict(fmt=2),
             dict(fmt=2, meta=(1 << 20) + 4), dict(n_pages=1 << 27),
             dict(n_pages=1 << 24, heads=64), dict(n_cells=1 << 22, n_pages=1 << 10)]


def _append(lk, pool, cells=(0, 1), rows=3, slots=FAKE, k=None, v=None, status=None):
    good = lk.loopkv_rows(1 << 20, 64, 128, 64)
    a = np.asarray(cells, np.int32)
    return lk.loopkv_paged_append(pool, a.ctypes.data_as(ctypes.c_void_p) if a.size else None,
                                  a.size, rows, slots, good if k is None else k,
                                  good if v is None else v, status, None)


def _bad_rows(lk):
    for kw in (dict(data=None), dict(data=(1 << 20) + 8), dict(cell_stride=-8),
               dict(row_stride=12), dict(head_stride=4)):
        yield lk.loopkv_rows(**{**dict(data=1 << 20, cell_stride=64, row_stride=128,
                                       head_stride=64), **kw})


def test_append_refuses_arguments(lk):
    assert _append(lk, None) == INVALID
    for kw in BAD_POOLS:
        assert _append(lk, _pool(lk, **kw)) == INVALID, kw
    pool = _pool(lk)
    assert _append(lk, pool, cells=()) == INVALID
    assert _append(lk, pool, cells=(0, 2)) == INVALID        # outside the pool
    assert _append(lk, pool, cells=(0, -2)) == INVALID
    assert _append(lk, pool, cells=(1, 1)) == INVALID        # listed twice
    assert _append(lk, _pool(lk, n_cells=300), cells=range(257)) == INVALID
    assert _append(lk, pool, rows=-1) == INVALID
    assert _append(lk, pool, slots=None) == INVALID
    assert _append(lk, pool, slots=ODD) == INVALID
    assert _append(lk, pool, status=ODD) == INVALID
    for rows in _bad_rows(lk):
        assert _append(lk, pool, k=rows) == INVALID
        assert _append(lk, pool, v=rows) == INVALID
    assert _append(lk, pool, rows=0, slots=None) == 0        # nothing to do
    assert _append(lk, pool, cells=(-1, -1)) == 0            # nothing is stored


def _decode(lk, pool, cells=(0, 1), current=None, batch=2, max_pages=4, group=2, sm_scale=0.0,
            table=FAKE, length=FAKE, q=None, cur=None, out=FAKE, lse=None, work=FAKE,
            nbytes=1 << 30, status=None):
    good = lk.loopkv_rows(1 << 20, 64, 128, 64)
    a = np.asarray(cells, np.int32)
    f = None if current is None else np.asarray(current, np.uint8)
    desc = lk.loopkv_paged_desc(batch, max_pages, group, sm_scale)
    return lk.loopkv_paged_decode(pool, desc, a.ctypes.data_as(ctypes.c_void_p) if a.size else None,
                                  None if f is None else f.ctypes.data_as(ctypes.c_void_p), a.size,
                                  table, length, good if q is None else q, cur, cur, out, lse, work,
                                  nbytes, status, None)


def test_decode_refuses_arguments(lk):
    assert _decode(lk, None) == INVALID
    for kw in BAD_POOLS:
        assert _decode(lk, _pool(lk, **kw)) == INVALID, kw
    pool = _pool(lk)
    for kw in (dict(batch=0), dict(batch=4097), dict(max_pages=0), dict(max_pages=(1 << 18) + 1),
               dict(group=0), dict(group=17), dict(sm_scale=float("nan")),
               dict(sm_scale=float("inf")), dict(cells=()), dict(cells=(0, 2)), dict(cells=(-1,)),
               dict(table=None), dict(table=ODD), dict(length=None), dict(length=ODD),
               dict(out=None), dict(out=ctypes.c_void_p((1 << 20) + 4)), dict(lse=ODD),
               dict(work=None), dict(work=ctypes.c_void_p((1 << 20) + 8)), dict(status=ODD),
               dict(nbytes=16), dict(current=(0, 1))):       # a current token without vectors
        assert _decode(lk, pool, **kw) == INVALID, kw
    for rows in _bad_rows(lk):
        assert _decode(lk, pool, q=rows) == INVALID
        assert _decode(lk, pool, current=(1, 1), cur=rows) == INVALID


def test_more_refusals(lk):
    # the new lengths in the place of the counts; a scale that 8-bit scores cannot carry
    other = ctypes.c_void_p((1 << 20) + 64)
    p = [FAKE, other, FAKE, FAKE, FAKE, FAKE, other, FAKE]
    assert _map(lk, ptrs=p) == INVALID
    pool = _pool(lk, fmt=2, meta=1 << 20)
    assert _decode(lk, pool, sm_scale=1e20) == INVALID


def test_workspace_is_what_decode_asks_for(lk):
    pool = _pool(lk)
    rc, nbytes = lk.loopkv_paged_workspace(pool, lk.loopkv_paged_desc(2, 4, 2, 0.0))
    assert rc == 0 and nbytes > 0
    assert _decode(lk, pool, nbytes=nbytes - 1) == INVALID
    assert lk.loopkv_paged_workspace(pool, lk.loopkv_paged_desc(2, 4, 17, 0.0))[0] == INVALID
    assert lk.loopkv_paged_workspace(None, lk.loopkv_paged_desc(2, 4, 2, 0.0))[0] == INVALID


def test_binding_refuses_before_the_library(lk):
    import torch
    from loop_aware_quantized_b200 import PagedCache, page_map, page_release, paged_append, paged_decode
    i32 = torch.zeros(2, dtype=torch.int32)
    table, one = torch.zeros((2, 4), dtype=torch.int32), torch.zeros(1, dtype=torch.int32)
    for call in (lambda: page_map(i32, i32, table, i32, one, 16, i32, torch.zeros(3, dtype=torch.int32)),
                 lambda: page_release(i32, i32, table, i32, one, 16),
                 lambda: page_map(i32, i32, table[0], i32, one, 16, i32, i32),
                 lambda: page_map(i32, i32, np.zeros((2, 4)), i32, one, 16, i32, i32),
                 lambda: page_map(i32, i32, table, i32, one, 16.5, i32, i32)):
        with pytest.raises(lk.LoopKVError) as e:
            call()
        assert e.value.status == INVALID
    pages = torch.zeros((1, 2, 2, 16, 64), dtype=torch.bfloat16)
    rows = torch.zeros((1, 2, 2, 64), dtype=torch.bfloat16)
    for call in (lambda: paged_append([0], rows, rows, i32, pages, pages),        # host tensors
                 lambda: paged_append([0], rows, rows, i32, pages.float(), pages.float()),
                 lambda: paged_append([0], rows, rows, i32, pages[0], pages[0]),
                 lambda: paged_decode([0], rows, pages, pages, table, i32),
                 lambda: paged_decode([0], rows, pages, pages, table[0], i32)):
        with pytest.raises(lk.LoopKVError) as e:
            call()
        assert e.value.status == INVALID
    for kw in (dict(shared=[2]), dict(shared=[-1]), dict(dtype=torch.float32), dict(max_batch=0),
               dict(max_pages=1 << 20), dict(n_loops=0)):
        with pytest.raises(lk.LoopKVError):
            PagedCache(**{**dict(n_loops=2, n_layers=2, n_kv_heads=2, head_dim=64, n_pages=4,
                                 page_size=16, max_batch=2, max_pages=4, device="cpu"), **kw})


def test_short_way_declines_what_it_does_not_handle(lk):
    # nothing but kNotPlain for arguments of any kind, and no error left behind
    import torch
    from loop_aware_quantized_b200 import _paged
    host = torch.zeros((2, 2), dtype=torch.int32)
    odd = [None, 0, -1, 1 << 70, 2.5, "x", b"x", [], [1 << 40], [True], (1, 2), np.zeros(3), np.zeros((2, 2), np.int32),
           np.arange(300), host, host[0], torch.zeros(3), torch.nn.Parameter(torch.zeros(2)), object()]
    for name, n in (("page_map", 12), ("page_release", 9), ("paged_append", 8), ("paged_decode", 14)):
        fn = getattr(_paged, name)
        assert fn() == -1 and fn(*[None] * (n + 1)) == -1
        for i in range(len(odd)):
            assert fn(*[odd[(i + j * 7) % len(odd)] for j in range(n)]) == -1
            assert fn(*[odd[i]] * n) == -1


def test_cache_maps_shared_cells_to_the_final_loop(lk):
    from loop_aware_quantized_b200 import PagedCache
    c = PagedCache(3, 2, 1, 64, 4, 16, 2, 4, shared=[0, 3], device="cpu")
    # stored: cells 1, 2, 4, 5 -> pool 0, 1, 2, 3; 0 reads layer 0's final cell, 3 layer 1's
    assert c.store_cell.tolist() == [-1, 0, 1, -1, 2, 3]
    assert c.pool_cell.tolist() == [2, 0, 1, 3, 2, 3]
    assert tuple(c.k_pages.shape) == (4, 4, 1, 16, 64)


def test_reference_map_by_hand():
    # page size 4; request 0 holds 3 tokens in page 7 and brings 2: one in page 7, one in a new
    # page (the free list's last, 5); request 1 is new with 4 tokens (page 2); request 2 brings 1
    # but only two pages were free
    table = np.array([[7, -1], [-1, -1], [-1, -1]])
    t, slots, starts, n, count, st = R.page_map(np.array([3, 0, 0]), np.array([2, 4, 1]), table,
                                                np.array([2, 5, 0, 0, 0, 0, 0, 0]), 2, 4, 9)
    assert slots.tolist() == [31, 20, 8, 9, 10, 11, -1, -1, -1]
    assert t.tolist() == [[7, 5], [2, -1], [-1, -1]]
    assert starts.tolist() == [0, 2, 6, 7] and n.tolist() == [5, 4, 0]
    assert count == 0 and st == R.NO_PAGES
    free, n, count, st = R.page_release(n, np.array([4, 0, 0]), t, np.zeros(8, np.int64), 0, 4)
    assert free[:2].tolist() == [5, 2] and n.tolist() == [4, 0, 0] and count == 2 and st == 0


def test_reference_decode_by_hand():
    # two tokens with scores 0 and ln 3: weights 1/4 and 3/4
    k = np.zeros((1, 1, 1, 2, 64))
    k[0, 0, 0, 1, 0] = np.log(3)
    v = np.zeros((1, 1, 1, 2, 64))
    v[0, 0, 0, 1, :] = 8.0
    q = np.zeros((1, 1, 1, 64))
    q[..., 0] = 1
    out, lse, _, _ = R.decode([0], q, k, v, None, np.array([[0]]), [2], 2, sm_scale=1.0)
    assert np.allclose(out, 6.0) and np.allclose(lse, np.log(4))
    # the same with the second token as the current one, and nothing stored of it
    k2, v2 = k.copy(), v.copy()
    k2[0, 0, 0, 1], v2[0, 0, 0, 1] = np.nan, np.nan
    cur = (k[:, :, :, 1], v[:, :, :, 1])
    out2, lse2, _, _ = R.decode([0], q, k2, v2, None, np.array([[0]]), [2], 2, cur=cur, sm_scale=1.0)
    assert np.array_equal(out, out2) and np.array_equal(lse, lse2)
    out, lse, _, _ = R.decode([0], q, k, v, None, np.array([[0]]), [0], 2)
    assert not out.any() and np.isneginf(lse).all()


def test_reference_quantizer_by_hand():
    x = np.array([[-1.0, 254.0, 0.0, 1.5], [3.0, 3.0, 3.0, 3.0], [0.0, 255.0, 0.5, 1.5]])
    code, scale, zero = R.quantize(x)
    assert code.tolist() == [[0, 255, 1, 2], [0, 0, 0, 0], [0, 255, 0, 2]]   # 2.5 -> 2, ties to even
    assert scale.tolist() == [1.0, 0.0, 1.0] and zero.tolist() == [-1.0, 3.0, 0.0]


def test_binding_declares_every_parameter(lk):
    # ctypes passes undeclared arguments as 32-bit ints: every parameter of the header is declared
    import os
    import re
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(root, "include", "loopkv.h")).read(), flags=re.S)
    found = 0
    for name, params in re.findall(r"\b(loopkv_\w+)\s*\(([^)]*)\)\s*;", text):
        found += 1
        n = len([x for x in params.split(",") if x.strip()])
        assert len(getattr(lk._lib, name).argtypes) == n, name
    assert found >= 18
