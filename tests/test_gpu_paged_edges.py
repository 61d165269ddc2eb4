"""Paged cells on the GPU at the ends of their ranges."""

import ctypes
import threading

import numpy as np
import pytest

from tests import paged_reference as R
from tests.test_gpu_paged import Case, check_map, empty_pool, host, ints, make_tables

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev(cuda_device):
    return cuda_device


# ------------------------------------------------------------ two threads

def at_once(calls, times):
    """Every call of ``calls`` ``times`` times, each in a thread of its own; their nonzero results."""
    found, gate = [[] for _ in calls], threading.Barrier(len(calls))

    def work(i):
        gate.wait()
        found[i] += [rc for rc in (calls[i]() for _ in range(times)) if rc]

    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(calls))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    return found


def test_decodes_of_two_threads(dev):
    # a small and the largest batch: the C calls run at once (ctypes drops the interpreter lock)
    import torch
    from loop_aware_quantized_b200 import loopkv as lk
    made = []
    for i, (batch, fmt) in enumerate(((1, "bf16"), (lk.LOOPKV_MAX_PAGED_BATCH, "bf16"))):
        c = Case(dev, fmt, [3] * min(batch, 2) + [0] * (batch - 2), heads=1, dim=128, ps=16, seed=i)
        table, n = ints(c.table, dev), ints(c.lengths, dev)
        out, stream = torch.zeros_like(c.q), torch.cuda.Stream(dev)
        pool = lk.loopkv_page_pool(*c.shape[:2], c.ps, 1, 128, lk.LOOPKV_PAGE_BF16, c.kp.data_ptr(), c.vp.data_ptr(), None)
        desc = lk.loopkv_paged_desc(batch, table.shape[1], 1, 0.0)
        rc, nbytes = lk.loopkv_paged_workspace(pool, desc)
        assert rc == 0
        work = torch.empty(nbytes, dtype=torch.uint8, device=dev)
        rows = lk.loopkv_rows(c.q.data_ptr(), 0, 0 if batch == 1 else 128, 0)
        cells = np.zeros(1, np.int32)
        args = (pool, desc, cells.ctypes.data_as(ctypes.c_void_p), None, 1, table.data_ptr(), n.data_ptr(), rows, None, None,
                out.data_ptr(), None, work.data_ptr(), nbytes, None, stream.cuda_stream)
        made.append((c, out, args, table, n, work, cells, stream))
    torch.cuda.synchronize()
    found = at_once([lambda a=m[2]: lk.loopkv_paged_decode(*a) for m in made], 3000)
    torch.cuda.synchronize()
    assert found == [[], []]
    for c, out, *_ in made:
        assert (out == c.run()[0]).all()


@pytest.mark.parametrize("call", ["map", "release"])
def test_page_calls_of_two_threads(dev, call):
    import torch
    from loop_aware_quantized_b200 import loopkv as lk
    made = []
    for batch in (3500, lk.LOOPKV_MAX_PAGED_BATCH):
        new, table = ints(np.zeros(batch), dev), ints(np.full((batch, 2), -1), dev)
        free, one = ints(np.arange(16), dev), ints([16], dev)
        slots, starts = ints(np.zeros(8), dev), ints(np.zeros(batch + 1), dev)
        n, n_out, one_out = ints(np.zeros(batch), dev), ints(np.full(batch, 5), dev), ints([0], dev)
        stream = torch.cuda.Stream(dev)
        p = {k: v.data_ptr() for k, v in dict(n=n, new=new, table=table, free=free, one=one, slots=slots, starts=starts,
                                             n_out=n_out, one_out=one_out).items()}
        if call == "map":
            args = (batch, 16, 2, 16, 8, p["n"], p["new"], p["table"], p["free"], p["one"], p["slots"], p["starts"], None,
                    p["n_out"], p["one_out"], None, stream.cuda_stream)
        else:
            args = (batch, 16, 2, 16, p["n"], p["new"], p["table"], p["free"], p["one"], p["n_out"], p["one_out"], None,
                    stream.cuda_stream)
        made.append((args, n_out, one_out, new, table, free, one, slots, starts, n, stream))
    torch.cuda.synchronize()
    fn = lk.loopkv_page_map if call == "map" else lk.loopkv_page_release
    found = at_once([lambda a=m[0]: fn(*a) for m in made], 3000)
    torch.cuda.synchronize()
    assert found == [[], []]
    assert all(not m[1].any() and int(m[2]) == 16 for m in made)


# ------------------------------------------------------- damaged bookkeeping

@pytest.mark.parametrize("bad", [-1, -2 ** 31, 1, 2 ** 31 - 1])
@pytest.mark.parametrize("batch,width", [(3, 4), (70, 5), (900, 9)])
@pytest.mark.parametrize("in_place", [False, True])
def test_release_with_a_count_out_of_range_hands_out_nothing(dev, bad, batch, width, in_place):
    # no page is pushed, and the count that is stored holds no page that a request still has
    from loop_aware_quantized_b200 import page_release
    rng = np.random.default_rng(batch)
    ps, n_pages = 8, batch * width
    if bad == 1:
        bad = n_pages + 1
    lengths = rng.integers(1, width * ps + 1, batch)
    table, free, _ = make_tables(rng, lengths, width, ps, n_pages)
    new = np.where(rng.random(batch) < 0.7, 0, lengths - 1)
    t = [ints(x, dev) for x in (lengths, new, table, free, [bad])]
    status = ints([0], dev)
    lo, co = (t[0], t[4]) if in_place else (ints(np.full(batch, 99), dev), ints([99], dev))
    page_release(*t, ps, lengths_out=None if in_place else lo, free_count_out=None if in_place else co, status=status)
    pushes = -(-lengths // ps) > -(-new // ps)
    assert np.array_equal(host(t[3]), free) and int(co) == 0
    assert np.array_equal(host(lo), np.where(pushes, lengths, new))
    assert int(status) == R.BAD_LENGTH | R.NO_PAGES
    check_map(dev, host(lo), np.full(batch, ps), host(t[2]), free, int(co), ps, batch * ps)


def test_decode_flags_every_page_id_outside_the_pool(dev):
    for fmt in ("bf16", "q8"):
        for ps in (16, 24):
            c = Case(dev, fmt, [100, 64, 20], heads=2, group=2, ps=ps, seed=40)
            for bad in (-2 ** 31, -2 ** 31 + 1, -1, c.shape[1], 2 ** 31 - 1):
                t = c.table.copy()
                t[0, 1] = bad
                c.check(table=t, status=R.BAD_PAGE)


# ------------------------------------------------------------------- weights

def dominated(dev, fmt, gap, value, n=512, batch=888, group=1):
    """Requests whose first token, of value 0, lies ``gap`` nats above the others, of value ``value``."""
    c = Case(dev, fmt, [n] * batch, heads=1, group=group, dim=64, ps=16, seed=50, width=n // 16)
    c.q.zero_()
    c.q[..., 0] = 1
    c.kp.zero_()
    c.vp.fill_(value)
    c.kp[0, c.table[:, 0], 0, 0, 0] = gap
    c.vp[0, c.table[:, 0], 0, 0] = 0
    return c


@pytest.mark.parametrize("group", [1, 8, 16])
@pytest.mark.parametrize("fmt,gap,value", [
    ("bf16", 300, 2.0 ** 120), ("bf16", 300, -2.0 ** 120), ("bf16", 75, 2.0 ** 100), ("bf16", 20, 2.0 ** 100),
    ("bf16", 300, 1.0), ("fp16", 300, 60000.0), ("fp16", 40, 60000.0), ("fp16", 40, -60000.0), ("fp16", 5, 60000.0)])
def test_decode_adds_nothing_for_weights_of_nothing(dev, fmt, gap, value, group):
    dominated(dev, fmt, gap, value, batch=888 if group == 1 else 50, group=group).check(sm_scale=1.0)


@pytest.mark.parametrize("gap", [14.0, 18.0, 22.0, 26.0])
def test_decode_fp16_weights_near_their_smallest_step(dev, gap):
    # a weight is kept to 2^-38 of the largest where that is more than 2^-16 of itself
    n, value = 512, 60000.0
    c = dominated(dev, "fp16", gap, value, n)
    out, lse, status = c.run(sm_scale=1.0)
    want = (n - 1) * np.exp(-gap) * value / (1 + (n - 1) * np.exp(-gap))
    tol, _ = R.bounds(np.full((1, 1), want), np.full((1, 1), want), np.full(1, gap), n, 2.0 ** -11)
    assert status == 0 and (np.abs(host(out).astype(np.float64) - want) <= tol + n * value * 2.0 ** -38).all()


@pytest.mark.parametrize("group", [1, 8, 16])
@pytest.mark.parametrize("fmt,gaps", [("bf16", (0, 1, 20, 80)), ("fp16", (0, 1, 10, 20, 25))])
def test_decode_keeps_infinite_values_infinite(dev, fmt, gaps, group):
    # at the largest weight, at middle ones, and at those next to the smallest that are kept
    for gap in gaps:
        for sign in (1, -1):
            c = dominated(dev, fmt, gap, 1.0, n=64, batch=5, group=group)
            c.vp[0, c.table[2, 1], 0, 3, 7] = sign * float("inf")
            c.vp[0, c.table[3, 0], 0, 0, 9] = sign * float("inf")
            out, _, _ = c.run(sm_scale=1.0)
            o = host(out)[0]
            assert (o[2, :, 7] == sign * np.inf).all() and (o[3, :, 9] == sign * np.inf).all()
            o[2, :, 7] = o[3, :, 9] = 0
            assert np.isfinite(o).all()


# -------------------------------------------------- 8-bit pages, any input

@pytest.mark.parametrize("dim", [64, 128])
def test_q8_append_keeps_the_trace_of_what_it_cannot_hold(dev, dim):
    # NaN, infinities and ranges beyond fp32: flagged, and the token decodes as NaN; its neighbours
    # are as they would be without it
    import torch
    from loop_aware_quantized_b200 import loopkv as lk, paged_append, paged_decode
    heads, ps, rows = 2, 8, 8
    g = torch.Generator(device=dev).manual_seed(dim)
    k, v, q = (torch.randn((1, rows, heads, dim), generator=g, device=dev).to(torch.bfloat16) for _ in range(3))
    top = torch.finfo(torch.bfloat16).max
    for part in (0, 1):
        for at in (0, dim // 2 + 3, dim - 1):
            for bad in (float("nan"), float("inf"), -float("inf"), "range"):
                kv = [k.clone(), v.clone()]
                if bad == "range":
                    kv[part][0, 5, 1, 1 - min(at, 1)], kv[part][0, 5, 1, at] = -top, top
                else:
                    kv[part][0, 5, 1, at] = bad
                kp, vp, meta = empty_pool(dev, "q8", (1, 1, heads, ps, dim))
                meta.zero_()
                status = ints([0], dev)
                paged_append([0], *kv, ints(np.arange(rows), dev), kp, vp, meta=meta, status=status)
                assert int(status) == lk.LOOPKV_PAGE_BAD_VALUE
                pages = host((kp, vp)[part])[0, 0]
                code, scale, zero = R.quantize(host((k, v)[part][0]))
                others = np.ones((heads, ps), bool)
                others[1, 5] = False
                assert np.array_equal(pages[others], code.transpose(1, 0, 2)[others]) and not pages[1, 5].any()
                out = host(paged_decode([0], q[:, :1], kp, vp, ints([[0]], dev), ints([rows], dev), meta=meta))
                assert np.isnan(out[0, 0, 1]).all() and np.isfinite(out[0, 0, 0]).all()


def test_q8_append_flags_value_ranges_that_decode_cannot_weigh(dev):
    # scales of values from 2^56 on; keys may have them
    import torch
    from loop_aware_quantized_b200 import loopkv as lk, paged_append, paged_decode
    x = torch.zeros((1, 3, 1, 64), dtype=torch.bfloat16, device=dev)
    q = torch.zeros((1, 1, 1, 64), dtype=torch.bfloat16, device=dev)
    for power, want in ((55, 0), (56, lk.LOOPKV_PAGE_BAD_VALUE)):
        big = x.clone()
        big[0, 1, 0, 5] = 255 * 2.0 ** power
        for kv, flag in (((x, big), want), ((big, x), 0)):
            kp, vp, meta = empty_pool(dev, "q8", (1, 1, 1, 4, 64))
            status = ints([0], dev)
            paged_append([0], *kv, ints([0, 1, 2], dev), kp, vp, meta=meta, status=status)
            assert int(status) == flag
            if flag == 0:  # equal scores: the mean of the three
                out = host(paged_decode([0], q, kp, vp, ints([[0]], dev), ints([3], dev), meta=meta))[0, 0, 0]
                ref = R.decode([0], host(q), host(kp), host(vp), host(meta), np.array([[0]]), [3], 4)
                tol, _ = R.bounds(ref[0], ref[2], ref[3], 3, 2.0 ** -8)
                assert (np.abs(out - ref[0][0, 0, 0]) <= tol[0, 0, 0]).all()


def test_q8_decode_reads_the_largest_queries(dev):
    # queries just below 2^64, key scales that bring their scores down
    c = Case(dev, "q8", [40, 7], heads=1, group=2, dim=64, seed=60)
    c.q.fill_(2.0 ** 64 * (1 - 2.0 ** -8))
    c.meta[..., 0] *= 2.0 ** -64
    c.meta[..., 1] = 0
    c.check()


# ----------------------------------------------------- arguments, both ways

def test_positive_scales_that_fp32_loses_are_refused(dev):
    # (a scale of 0 means 1 / sqrt(head dim))
    import torch
    from loop_aware_quantized_b200 import paged_decode
    from loop_aware_quantized_b200.loopkv import LoopKVError
    c = Case(dev, "bf16", [10, 20], heads=2, group=2, dim=64, seed=61)
    t, n = ints(c.table, dev), ints(c.lengths, dev)
    for stream in (None, torch.cuda.current_stream()):
        for scale in (1e-50, 2.0 ** -150, 1e300):
            with pytest.raises(LoopKVError) as e:
                paged_decode([0], c.q, c.kp, c.vp, t, n, sm_scale=scale, stream=stream)
            assert e.value.status == 1
    c.check(sm_scale=2.0 ** -126)


def test_flags_are_truth_values(dev):
    import torch
    from loop_aware_quantized_b200 import paged_decode
    c = Case(dev, "bf16", [10, 20], heads=2, group=2, dim=64, cells=(0, 0, 0, 0), seed=62)
    args = (c.cells, c.q, c.kp, c.vp, ints(c.table, dev), ints(c.lengths, dev))
    want = paged_decode(*args, cur_k=c.cur[0], cur_v=c.cur[1], current=[True, False, True, True])
    assert (want[0] != want[1]).any()
    for flags in (np.array([256, 0, 512, -256]), [256, 0, 2 ** 40, 0.25], np.array([0.5, 0.0, 1e-9, -1.0])):
        assert (paged_decode(*args, cur_k=c.cur[0], cur_v=c.cur[1], current=flags) == want).all()


def test_what_one_way_refuses_the_other_does(dev):
    # the compiled checks (the current stream) and those in Python (a stream given): every bad
    # argument fails on both, and the first way leaves it to the second or names the same error
    import torch
    from loop_aware_quantized_b200 import _paged, page_map, page_release, paged_append, paged_decode
    from loop_aware_quantized_b200.loopkv import LoopKVError
    c = Case(dev, "q8", [10, 20], heads=2, group=2, dim=64, seed=63)
    t, n = ints(c.table, dev), ints(c.lengths, dev)
    i2, one, s2 = ints([1, 1], dev), ints([2], dev), ints([1, 2], dev)
    free = ints(np.arange(c.shape[1]), dev)
    wide = torch.zeros((1, 2, 2, 68), dtype=torch.bfloat16, device=dev)
    vec, vec4 = c.cur[0], c.q
    calls = {
        "page_map": (page_map, dict(lengths=n, n_new=i2, table=t, free=free, free_count=one, page_size=16, slots=s2,
                                    starts=ints([0] * 3, dev), newest=None, lengths_out=None, free_count_out=None, status=None)),
        "page_release": (page_release, dict(lengths=n, new_lengths=n.clone(), table=t, free=free, free_count=one, page_size=16,
                                            lengths_out=None, free_count_out=None, status=None)),
        "paged_append": (paged_append, dict(cells=[0], k=vec, v=vec, slots=s2, k_pages=c.kp, v_pages=c.vp, meta=c.meta,
                                            status=None)),
        "paged_decode": (paged_decode, dict(cells=[0], q=vec4, k_pages=c.kp, v_pages=c.vp, table=t, lengths=n, meta=c.meta,
                                            cur_k=None, cur_v=None, current=None, out=None, lse=None, sm_scale=0.0,
                                            status=None)),
    }
    ints_bad = [n.long(), n.float(), n[:1], n.cpu(), ints([0] * 4, dev)[::2], ints([0] * 3, dev), t]
    vec_bad = [vec.half(), vec.float(), vec[..., :32], vec[:, :1], wide[..., 2:66], wide[..., :64], vec[0], vec.cpu()]
    pages_bad = [c.kp.to(torch.int32), c.kp[0], c.kp[..., :32], c.kp[:, :0], c.kp.cpu(), c.kp.transpose(1, 2)]
    bad = {
        "lengths": ints_bad, "n_new": ints_bad, "new_lengths": ints_bad, "lengths_out": ints_bad, "newest": ints_bad,
        "table": [t.long(), t.t(), t[0], t[:1], t[:, :0], t.cpu()], "free": [free.long(), t, free.cpu(), free[:0]],
        "free_count": [i2, one.long(), one.cpu()], "free_count_out": [i2, one.long(), one.cpu()],
        "status": [i2, one.long(), one.cpu()], "starts": [n, ints([0] * 4, dev), ints([0] * 3, dev).long()],
        "page_size": [0, -1, 1025, 16.5, True, 1 << 40], "k": vec_bad, "v": vec_bad, "cur_k": vec_bad + [vec], "cur_v": vec_bad + [vec],
        "q": [vec4.half(), vec4[..., :32], vec4[:, :1], vec4[:, :, :3], vec4.cpu(), wide[..., 2:66]],
        "k_pages": pages_bad, "v_pages": pages_bad, "meta": [None, c.meta.half(), c.meta[..., :3], c.meta.cpu()],
        "cells": [[], [1], [-2], [0, 0], [2 ** 32], list(range(300)), np.array([2 ** 32]), np.array([[0.5]])],
        "current": [[True], np.array([1], np.uint8), [True, False]], "out": [vec4.float(), vec4[:, :, :2], vec4.cpu(), vec4.half()],
        "lse": [torch.zeros(3, device=dev), torch.zeros((1, 2, 4), device=dev).double()],
        "sm_scale": [float("nan"), float("inf"), 1e300, 1e20],
        "slots": [s2.long(), s2.cpu(), t],
    }
    before = [x.clone() for x in (c.kp, c.vp, t, n, free, one)]
    tried = 0
    for name, (fn, good) in calls.items():
        short = getattr(_paged, name)
        for arg in good:
            for x in bad[arg]:
                kw = {**good, arg: x}
                got = short(*kw.values())
                assert got in (-1, 1), (name, arg, x)
                for stream in (None, torch.cuda.current_stream()):
                    with pytest.raises(LoopKVError) as e:
                        fn(**kw, stream=stream)
                    assert e.value.status == 1, (name, arg, x)
                tried += 1
    torch.cuda.synchronize()
    assert tried > 150 and all((a == b).all() for a, b in zip(before, (c.kp, c.vp, t, n, free, one)))


# -------------------------------------------------------------- many blocks

def test_page_map_refuses_on_many_blocks(dev):
    # refused requests of every kind among admitted ones, rows just above what one block takes
    ps, width = 8, 40
    for rows, batch in ((256, 60), (257, 60), (3000, 60), (9000, 700), (9000, 2500)):
        rng = np.random.default_rng(rows + batch)
        lengths = rng.integers(0, 100, batch)
        new = np.bincount(rng.integers(0, batch, rows), minlength=batch)
        table, free, count = make_tables(rng, lengths, width, ps, batch * width)
        lengths[3], new[7], lengths[11], new[20] = -5, -2, 2 ** 31 - 1, 2 ** 31 - 1
        table[1, :13] = batch * width                    # held pages outside the pool
        free[count - 3:count - 1] = -1
        need = int(np.maximum(0, new[:18]).sum()) // ps + 20
        for in_place in (False, True):
            st = check_map(dev, lengths, new, table, free, count, ps, rows, in_place)[5]
            assert st & R.BAD_LENGTH and st & R.NO_TABLE and st & R.NO_ROWS
            check_map(dev, lengths, np.minimum(new, 500), table, free, min(need, count), ps, rows + 1000, in_place)


@pytest.mark.parametrize("n_pages", [255, 256, 257, 4095, 4096, 4097, 20000])
@pytest.mark.parametrize("in_place", [False, True])
def test_page_release_refuses_on_any_number_of_blocks(dev, n_pages, in_place):
    # one block takes 256 pages, in place 4096: bad lengths, bad entries, a list that is nearly full
    from loop_aware_quantized_b200 import page_release
    rng = np.random.default_rng(n_pages)
    batch = 40
    width = -(-n_pages // batch) + 1
    lengths = rng.integers(0, n_pages // batch + 1, batch)
    table, free, count = make_tables(rng, lengths, width, 1, n_pages)
    new = np.where(rng.random(batch) < 0.8, 0, lengths // 2)
    for case in ("plain", "bad", "nearly full", "full"):
        n, a, tab, cnt = lengths.copy(), new.copy(), table.copy(), count
        if case != "plain":
            n[2], a[5], a[9], n[13] = -1, -1, n[9] + 1, width + 1
            tab[20, :n[20]] = n_pages
            tab[21, :n[21] // 2] = -9
        if case == "nearly full":
            cnt = n_pages - int((n[:12] - a[:12]).clip(0).sum()) - 1
        if case == "full":
            cnt = n_pages
        t = [ints(x, dev) for x in (n, a, tab, free, [cnt])]
        lo, co = (t[0], t[4]) if in_place else (ints(np.full(batch, 99), dev), ints([99], dev))
        status = ints([0], dev)
        page_release(*t, 1, lengths_out=None if in_place else lo, free_count_out=None if in_place else co, status=status)
        f, out, c, st = R.page_release(n, a, tab, free, cnt, 1)
        assert np.array_equal(host(t[3]), f) and np.array_equal(host(lo), out) and int(co) == c and int(status) == st, case
        assert np.array_equal(host(t[2]), tab)


# ------------------------------------------------------------ largest sizes

@pytest.mark.parametrize("fmt", ["bf16", "fp16", "q8"])
def test_decode_of_the_largest_scores(dev, fmt):
    # scores of 2^23 and -2^23, exact in fp32: the one above the others by 2^10 takes all the weight,
    # equal ones share it
    import torch
    for sign in (1, -1):
        c = Case(dev, fmt, [48, 16, 1], heads=2, group=2, dim=64, ps=16, seed=70, width=3)
        c.q.fill_(2.0 ** 11)
        if fmt == "q8":
            c.kp.fill_(128)
            c.meta[..., 0], c.meta[..., 1] = sign * 2.0 ** 4, 0
        else:
            c.kp.fill_(sign * 2.0 ** 11)
        # <q, k> = 64 * 2^11 * 2^11 = 2^28; the first request's token 20 has 64 * 2^11 * 8 = 2^20 more
        page = int(c.table[0, 1])
        if fmt == "q8":
            c.meta[0, page, :, 4, 1] += 8.0
        else:
            c.kp[0, page, :, 4] += 2.0 ** 3 if fmt == "fp16" else 2.0 ** 4  # (a step of bf16 is 8 below, 16 above 2^11)
        out, lse, status = c.run(sm_scale=2.0 ** -5)
        o, e = host(out).astype(np.float64)[0], host(lse)[0]
        v, size = R.stored(host(c.vp), None if c.meta is None else host(c.meta), 2)
        for b, n in enumerate(c.lengths):
            pos = np.arange(n) if b else np.array([20])
            want, around = (x[0, c.table[b, pos // 16], :, pos % 16].mean(0).repeat(2, 0) for x in (v, size))
            # weights to 2^-16, twice over with their sum, and the output's rounding
            assert (np.abs(o[b] - want) <= 2.0 ** -14 * around + (2.0 ** -11 if fmt == "fp16" else 2.0 ** -8) * np.abs(want)).all()
        assert status == 0 and (np.abs(np.abs(e) - 2.0 ** 23) <= 2.0 ** 17).all()


def test_decode_of_the_most_heads_and_cells(dev):
    # 65536 heads of one request; 256 listed cells, apart and shared
    import torch
    from loop_aware_quantized_b200 import paged_append, paged_decode
    heads = 1 << 16
    g = torch.Generator(device=dev).manual_seed(71)
    k, v, q = (torch.randn((1, 2, heads, 64), generator=g, device=dev).to(torch.bfloat16) for _ in range(3))
    kp, vp = (torch.zeros((1, 3, heads, 1, 64), dtype=torch.bfloat16, device=dev) for _ in range(2))
    paged_append([0], k, v, ints([2, 0], dev), kp, vp)
    out = paged_decode([0], q, kp, vp, ints([[2], [0]], dev), ints([1, 1], dev))
    assert (out == v).all()                              # one token each: its value
    cells = 256
    k, v, q = (torch.randn((cells, 2, 3, 64), generator=g, device=dev).to(torch.bfloat16) for _ in range(3))
    kp, vp = (torch.zeros((cells, 3, 3, 1, 64), dtype=torch.bfloat16, device=dev) for _ in range(2))
    order = np.random.default_rng(0).permutation(cells)
    paged_append(order, k, v, ints([2, 0], dev), kp, vp)
    t, n = ints([[2], [0]], dev), ints([1, 1], dev)
    assert (paged_decode(order, q, kp, vp, t, n) == v).all()
    at = int(order[5])
    assert (paged_decode([at] * cells, q, kp, vp, t, n) == v[5]).all()
    assert (paged_decode([at] * cells, q, kp, vp, t, n, cur_k=k, cur_v=v) == v).all()


@pytest.mark.parametrize("fmt,dim,group", [("bf16", 64, 1), ("fp16", 64, 4), ("q8", 128, 8), ("bf16", 128, 16)])
def test_decode_repeats_itself_bit_for_bit(dev, fmt, dim, group):
    # split units, their joins, other work on the GPU between: the order of sums does not change
    import torch
    c = Case(dev, fmt, [50000, 3, 0, 700, 7001], heads=2, group=group, dim=dim, ps=16, seed=72)
    first = c.run()
    side, x = torch.cuda.Stream(dev), torch.randn((2048, 2048), device=dev)
    for i in range(20):
        if i % 2:
            with torch.cuda.stream(side):
                x = torch.tanh(x @ x)
        again = c.run()
        assert (first[0] == again[0]).all() and (first[1] == again[1]).all()
