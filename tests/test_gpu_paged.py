"""Paged cells on the GPU against their plain 64-bit forms
(``tests/paged_reference.py``): bookkeeping and codes bit for bit, attention
within the bounds that its roundings allow."""

import numpy as np
import pytest

from tests import paged_reference as R

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev(cuda_device):
    return cuda_device


def ints(a, dev):
    import torch
    return torch.tensor(np.asarray(a), dtype=torch.int32, device=dev)


def host(t):
    import torch
    if t.dtype == torch.bfloat16:
        return t.float().cpu().numpy()
    return t.cpu().numpy()


# ------------------------------------------------------------------ page_map

def make_tables(rng, lengths, width, ps, n_pages, slack=None):
    """Random pages for the held tokens (garbage behind them), the rest free."""
    order = rng.permutation(n_pages)
    table = rng.integers(-5, n_pages + 5, (len(lengths), width))
    used = 0
    for b, n in enumerate(lengths):
        held = -(-max(int(n), 0) // ps)
        if held <= width:
            table[b, :held] = order[used:used + held]
            used += held
    free = np.full(n_pages, -7)
    free[:n_pages - used] = order[used:]
    return table, free, n_pages - used


def run_map(dev, lengths, new, table, free, count, ps, rows, in_place=False):
    import torch
    from loop_aware_quantized_b200 import page_map
    t = [ints(x, dev) for x in (lengths, new, table, free, [count])]
    slots, starts = ints(np.full(rows, 99), dev), ints(np.zeros(len(lengths) + 1), dev)
    newest, status = ints(np.full(len(lengths), 99), dev), ints([0], dev)
    lo, co = (t[0], t[4]) if in_place else (ints(np.full(len(lengths), 99), dev), ints([99], dev))
    page_map(*t, ps, slots, starts, newest=newest, lengths_out=None if in_place else lo,
             free_count_out=None if in_place else co, status=status)
    torch.cuda.synchronize()
    assert np.array_equal(host(t[3]), free) and np.array_equal(host(t[1]), new)
    return host(t[2]), host(slots), host(starts), host(lo), int(co), int(status), host(newest)


def check_map(dev, lengths, new, table, free, count, ps, rows, in_place=False):
    got = run_map(dev, lengths, new, table, free, count, ps, rows, in_place)
    want = R.page_map(np.asarray(lengths), np.asarray(new), table, free, count, ps, rows)
    for name, g, w in zip(("table", "slots", "starts", "lengths", "count", "status"), got, want):
        assert np.array_equal(g, w), name
    newest = [int(want[1][want[2][b + 1] - 1]) if want[3][b] > max(lengths[b], 0) else -1
              for b in range(len(lengths))]
    assert got[6].tolist() == newest
    return want


@pytest.mark.parametrize("batch,ps,ctx,mode,short", [
    (1, 16, 0, "prompt", False), (1, 1, 40, "step", False), (3, 24, 100, "step", False),
    (32, 64, 2000, "step", False), (33, 16, 300, "chunk", False), (255, 7, 90, "chunk", True),
    (256, 16, 0, "prompt", False), (1025, 16, 64, "chunk", False), (4096, 32, 100, "step", True),
    (4095, 1, 3, "chunk", False), (17, 1024, 5000, "chunk", True)])
@pytest.mark.parametrize("in_place", [False, True])
def test_page_map(dev, batch, ps, ctx, mode, short, in_place):
    rng = np.random.default_rng(batch * 31 + ps)
    lengths = rng.integers(0, ctx + 1, batch)
    if mode == "step":
        new = (rng.random(batch) < 0.8).astype(int)
    else:
        new = np.where(rng.random(batch) < 0.5, rng.integers(0, 900, batch), 0)
    rows = int(new.sum()) + 13
    width = -(-(ctx + 900) // ps) + 1
    n_pages = sum(-(-(n + a) // ps) for n, a in zip(lengths, new)) + 3
    table, free, count = make_tables(rng, lengths, width, ps, n_pages)
    if short:
        count = max(0, count // 2)
    want = check_map(dev, lengths, new, table, free, count, ps, rows, in_place)
    assert bool(want[5] & R.NO_PAGES) == short


def test_page_map_boundaries(dev):
    # every length against every count around a page's end
    ps, rng = 4, np.random.default_rng(1)
    lengths, new = (x.reshape(-1) for x in np.meshgrid(np.arange(10), np.arange(10)))
    table, free, count = make_tables(rng, lengths, 8, ps, 600)
    check_map(dev, lengths, new, table, free, count, ps, int(new.sum()))


def test_page_map_refusals(dev):
    ps, width = 8, 4
    lengths = np.array([3, -1, 30, 5, 8, 0, 2 ** 31 - 1, 1, 0, 7])
    new = np.array([2, 1, 3, -4, 9, 0, 2 ** 31 - 1, 40, 2 ** 30, 1])
    rng = np.random.default_rng(2)
    table, free, count = make_tables(rng, np.clip(lengths, 0, 32) * (lengths < 100), width, ps, 40)
    for rows in (60, 15, 1):
        want = check_map(dev, lengths, new, table, free, count, ps, rows)
        assert want[5] & (R.BAD_LENGTH | R.NO_TABLE | R.NO_ROWS)
    # a free count out of range gives no page
    for bad in (-1, 41):
        assert check_map(dev, lengths, new, table, free, bad, ps, 60)[5] & R.BAD_LENGTH
    # page ids outside the pool: of the partly filled page, of the free list
    t2, f2 = table.copy(), free.copy()
    t2[0, 0], f2[count - 1] = 40, -3
    assert check_map(dev, lengths, new, t2, f2, count, ps, 60)[5] & R.BAD_PAGE


def test_page_map_without_rows(dev):
    # a step that brings nothing, and one whose tokens find no row
    rng = np.random.default_rng(6)
    lengths = np.array([5, 0, 16, 31])
    table, free, count = make_tables(rng, lengths, 3, 16, 9)
    assert check_map(dev, lengths, np.zeros(4, int), table, free, count, 16, 0)[5] == 0
    assert check_map(dev, lengths, np.array([0, 0, 1, 0]), table, free, count, 16, 0)[5] == R.NO_ROWS
    check_map(dev, lengths, np.zeros(4, int), table, free, count, 16, 3, in_place=True)


def test_page_map_long_prompts(dev):
    # a cluster's rows, more than one chunk per warp, one giant request among small ones
    rng = np.random.default_rng(3)
    new = np.concatenate([rng.integers(0, 3, 100), [200001], rng.integers(0, 5000, 30), np.zeros(50, int)])
    lengths = rng.integers(0, 50, new.size)
    ps, rows = 16, int(new.sum()) + 5000
    n_pages = int((-(-(lengths + new) // ps)).sum())
    table, free, count = make_tables(rng, lengths, -(-200100 // ps), ps, n_pages)
    check_map(dev, lengths, new, table, free, count, ps, rows)


@pytest.mark.parametrize("batch,ps,ctx", [(1, 1, 1), (3, 24, 100), (64, 16, 4000), (1024, 16, 700),
                                          (4096, 5, 40)])
@pytest.mark.parametrize("in_place", [False, True])
def test_page_release(dev, batch, ps, ctx, in_place):
    import torch
    from loop_aware_quantized_b200 import page_release
    rng = np.random.default_rng(batch)
    lengths = rng.integers(0, ctx + 1, batch)
    width = -(-ctx // ps) + 1
    n_pages = int((-(-lengths // ps)).sum()) + 2
    table, free, count = make_tables(rng, lengths, width, ps, n_pages)
    new = np.where(rng.random(batch) < 0.4, 0, np.maximum(0, lengths - rng.integers(0, 2 * ps, batch)))
    t = [ints(x, dev) for x in (lengths, new, table, free, [count])]
    status = ints([0], dev)
    lo, co = (t[0], t[4]) if in_place else (ints(np.zeros(batch), dev), ints([0], dev))
    page_release(*t, ps, lengths_out=None if in_place else lo, free_count_out=None if in_place else co,
                 status=status)
    torch.cuda.synchronize()
    f, n, c, st = R.page_release(lengths, new, table, free, count, ps)
    assert np.array_equal(host(t[3]), f) and np.array_equal(host(lo), n)
    assert int(co) == c and int(status) == st == 0 and np.array_equal(host(t[2]), table)


def test_page_release_refusals(dev):
    from loop_aware_quantized_b200 import page_release
    lengths = np.array([9, 5, -2, 100, 16, 8, 31])
    new = np.array([10, -1, 0, 0, 3, 0, 0])
    rng = np.random.default_rng(5)
    table, free, count = make_tables(rng, np.clip(lengths, 0, 32) * (lengths < 99), 4, 8, 24)
    for cnt, tab in ((count, table), (22, table), (24, table), (-1, table), (25, table),
                     (count, np.where(table == table[4, 1], 24, table))):
        t = [ints(x, dev) for x in (lengths, new, tab, free, [cnt])]
        status = ints([0], dev)
        page_release(*t, 8, status=status)
        f, n, c, st = R.page_release(lengths, new, tab, free, cnt, 8)
        assert np.array_equal(host(t[3]), f) and np.array_equal(host(t[0]), n)
        assert int(t[4]) == c and int(status) == st and st & R.BAD_LENGTH


def test_page_calls_around_a_few_hundred_rows(dev):
    # one block or many, 256 to 1024 threads, outputs apart or in place
    for batch, rows in ((30, 255), (30, 256), (30, 257), (513, 256), (513, 600), (512, 1500), (2048, 300),
                        (2049, 300), (2049, 3000)):
        rng = np.random.default_rng(batch + rows)
        lengths = rng.integers(0, 50, batch)
        new = np.bincount(rng.integers(0, batch, rows), minlength=batch)
        n_pages = int((-(-(lengths + new) // 8)).sum()) + 2
        table, free, count = make_tables(rng, lengths, int((lengths + new).max()) // 8 + 1, 8, n_pages)
        for in_place in (False, True):
            check_map(dev, lengths, new, table, free, count, 8, rows, in_place)
            check_map(dev, lengths, new, table, free, count // 2, 8, rows, in_place)


# --------------------------------------------------------------- paged_append

def torch_dtype(fmt):
    import torch
    return {"bf16": torch.bfloat16, "fp16": torch.float16, "q8": torch.uint8}[fmt]


def vector_dtype(fmt):
    import torch
    return torch.float16 if fmt == "fp16" else torch.bfloat16


def empty_pool(dev, fmt, shape, seed=0):
    """Pages full of a pattern, so that every byte written elsewhere shows."""
    import torch
    g = torch.Generator(device=dev).manual_seed(seed)
    raw = lambda s, n: torch.randint(0, 256, s[:-1] + (s[-1] * n,), generator=g, device=dev,  # noqa: E731
                                     dtype=torch.uint8)
    n = 1 if fmt == "q8" else 2
    k, v = (raw(shape, n).view(torch_dtype(fmt)) for _ in range(2))
    meta = raw(shape[:4] + (4,), 4).view(torch.float32) if fmt == "q8" else None
    return k, v, meta


def as_bytes(t):
    import torch
    return None if t is None else t.contiguous().view(torch.uint8).cpu().numpy()


@pytest.mark.parametrize("fmt", ["bf16", "fp16", "q8"])
@pytest.mark.parametrize("cells,rows,heads,dim,ps", [
    ([0], 1, 1, 64, 16), ([1, 0], 3, 2, 128, 24), ([2, -1, 0], 33, 5, 64, 1),
    ([1], 700, 3, 128, 64), ([0, 1, 2], 37, 16, 128, 7)])
def test_paged_append(dev, fmt, cells, rows, heads, dim, ps):
    import torch
    from loop_aware_quantized_b200 import paged_append
    g = torch.Generator(device=dev).manual_seed(rows)
    n_pages = -(-rows // ps) + 2
    shape = (3, n_pages, heads, ps, dim)
    kp, vp, meta = empty_pool(dev, fmt, shape)
    want = [as_bytes(x) for x in (kp, vp, meta)]
    dt = vector_dtype(fmt)
    k = torch.randn((len(cells), rows, heads, dim), generator=g, device=dev).to(dt)
    v = (3 * torch.randn((len(cells), rows, heads, dim), generator=g, device=dev) - 1).to(dt)
    k[:, 0, 0] = 2.5                                     # a vector without a range
    v[:, rows // 2, -1].clamp_(min=0)
    slots = np.random.default_rng(rows).permutation(n_pages * ps)[:rows]
    slots[rows // 3::5] = -1
    if rows > 4:
        slots[1], slots[2] = n_pages * ps, -2            # outside the pool: skipped and flagged
    status = ints([0], dev)
    paged_append(cells, k, v, ints(slots, dev), kp, vp, meta=meta, status=status)
    torch.cuda.synchronize()
    assert int(status) == (R.BAD_SLOT if rows > 4 else 0)
    for i, c in enumerate(cells):
        for part, (x, out) in enumerate(((k, want[0]), (v, want[1]))):
            vec = x[i].float().cpu().numpy()
            raw = x[i].view(torch.uint8).cpu().numpy()
            code, scale, zero = R.quantize(vec)
            for r, s in enumerate(slots):
                if c < 0 or not 0 <= s < n_pages * ps:
                    continue
                page, off = divmod(int(s), ps)
                out[c, page, :, off] = code[r] if fmt == "q8" else raw[r]
                if fmt == "q8":
                    m = np.stack([scale[r], zero[r]], -1).astype(np.float32)
                    want[2][c, page, :, off, 8 * part:8 * part + 8] = m.view(np.uint8)
    for name, g_, w in zip(("k", "v", "meta"), (kp, vp, meta), want):
        if w is not None:
            assert np.array_equal(as_bytes(g_), w), name


@pytest.mark.parametrize("dim", [64, 128])
def test_paged_append_q8_codes_at_their_borders(dev, dim):
    # quotients on and next to half steps, ranges from subnormal to huge: the codes of the
    # definition, bit for bit
    import torch
    from loop_aware_quantized_b200 import paged_append
    rng = np.random.default_rng(dim)
    rows, heads = 600, 2
    x = rng.standard_normal((2, rows, heads, dim))
    x[:, :100] = rng.integers(-127, 128, (2, 100, heads, dim))
    x[:, :100, :, 0], x[:, :100, :, 1] = -127.5, 127.5             # scale 1: halves everywhere
    x[:, 100:200] = rng.integers(-20, 21, (2, 100, heads, dim)) / 2.0
    x[:, 200:500] *= 10.0 ** rng.uniform(-38, 37, (2, 300, heads, 1))
    x[:, 500:520] = rng.integers(-3, 4, (2, 20, heads, dim)) * 2.0 ** -133  # subnormal ranges
    x[:, 520:540, :, 1:] = 0                                       # one value apart from the rest
    x[:, 540:560] = np.where(rng.random((2, 20, heads, dim)) < 0.5, 0.0, -0.0)
    x = torch.tensor(x, dtype=torch.float32, device=dev).to(torch.bfloat16)
    ps = 16
    kp, vp, meta = empty_pool(dev, "q8", (1, -(-rows // ps), heads, ps, dim))
    paged_append([0], x[:1], x[1:], ints(np.arange(rows), dev), kp, vp, meta=meta)
    flat = lambda t: host(t[0].transpose(1, 2).reshape(-1, heads, t.shape[-1])[:rows])  # noqa: E731
    for part, (vec, pages) in enumerate(((x[0], kp), (x[1], vp))):
        code, scale, zero = R.quantize(host(vec))
        assert np.array_equal(flat(pages), code)
        got = flat(meta)[..., 2 * part:2 * part + 2]
        assert np.array_equal(got.view(np.uint32), np.stack([scale, zero], -1).view(np.uint32))


def test_page_calls_around_the_one_block_limit(dev):
    # rows (map) and pages (release) just below, at and above what one block takes
    for rows in (1, 1023, 1024, 1025, 4095, 4096, 4097, 5000):
        rng = np.random.default_rng(rows)
        lengths = rng.integers(0, 30, 40)
        new = np.bincount(rng.integers(0, 40, rows), minlength=40)
        n_pages = int((-(-(lengths + new) // 4)).sum()) + 1
        table, free, count = make_tables(rng, lengths, int((lengths + new).max()) // 4 + 1, 4, n_pages)
        for in_place in (False, True):
            check_map(dev, lengths, new, table, free, count, 4, rows, in_place)
    from loop_aware_quantized_b200 import page_release
    for n_pages in (4096, 4097, 9000):
        rng = np.random.default_rng(n_pages)
        lengths = rng.integers(0, n_pages // 64, 64)
        table, free, count = make_tables(rng, lengths, n_pages, 1, n_pages)
        new = np.where(rng.random(64) < 0.8, 0, lengths // 2)
        t = [ints(x, dev) for x in (lengths, new, table, free, [count])]
        page_release(*t, 1, lengths_out=t[1])            # the new lengths' own memory
        f, n, c, st = R.page_release(lengths, new, table, free, count, 1)
        assert np.array_equal(host(t[3]), f) and np.array_equal(host(t[1]), n) and int(t[4]) == c


def test_paged_append_reads_strided_vectors(dev):
    import torch
    from loop_aware_quantized_b200 import paged_append
    heads, dim, rows, ps = 3, 64, 21, 8
    fused = torch.randn((rows, 2, 3 * heads, dim), device=dev).to(torch.bfloat16)  # [rows, cells, q|k|v heads]
    k, v = (fused[:, :, a * heads:(a + 1) * heads].transpose(0, 1) for a in (1, 2))
    slots = ints(np.arange(rows)[::-1] + 2, dev)
    pools = [empty_pool(dev, "bf16", (2, 4, heads, ps, dim)) for _ in range(2)]
    paged_append([1, 0], k, v, slots, *pools[0][:2])
    paged_append([1, 0], k.contiguous(), v.contiguous(), slots, *pools[1][:2])
    for a, b in zip(*pools):
        assert a is None or np.array_equal(as_bytes(a), as_bytes(b))


# --------------------------------------------------------------- paged_decode

class Case:
    """Pages, table and queries of a decode; pages behind the lengths are NaN."""

    def __init__(self, dev, fmt, lengths, heads=2, group=1, dim=64, ps=16, cells=(0,), n_cells=None,
                 seed=0, width=None, scale=1.0):
        import torch
        rng = np.random.default_rng(seed)
        g = torch.Generator(device=dev).manual_seed(seed)
        self.fmt, self.ps, self.cells, self.group = fmt, ps, list(cells), group
        self.heads, self.dim, self.batch = heads, dim, len(lengths)
        self.lengths = np.asarray(lengths)
        held = -(-np.maximum(self.lengths, 0) // ps)
        width = int(max(1, held.max())) + 1 if width is None else width
        n_pages = int(held.sum()) + 2
        self.table, _, _ = make_tables(rng, self.lengths, width, ps, n_pages)
        self.shape = (n_cells or max(cells) + 1, n_pages, heads, ps, dim)
        dt = vector_dtype(fmt)
        randn = lambda *s: torch.randn(s, generator=g, device=dev)  # noqa: E731
        self.meta = None
        if fmt == "q8":
            self.kp, self.vp = (torch.randint(0, 256, self.shape, generator=g, device=dev,
                                              dtype=torch.uint8) for _ in range(2))
            m = torch.rand(self.shape[:4] + (4,), generator=g, device=dev)
            m[..., 0::2] = 0.01 + 0.01 * m[..., 0::2]
            m[..., 1::2] = -100 * m[..., 0::2] - m[..., 1::2]
            self.meta = m
        else:
            self.kp, self.vp = randn(*self.shape).to(dt), randn(*self.shape).to(dt)
        for b, n in enumerate(self.lengths):          # what lies behind a request's last token
            if n > 0 and n % ps:
                page = self.table[b, n // ps]
                if self.meta is None:
                    self.kp[:, page, :, n % ps:] = float("nan")
                    self.vp[:, page, :, n % ps:] = float("inf")
                else:
                    self.meta[:, page, :, n % ps:] = float("nan")
        self.q = (scale * randn(len(cells), self.batch, heads * group, dim)).to(dt)
        self.cur = tuple(randn(len(cells), self.batch, heads, dim).to(dt) for _ in range(2))
        self.dev = dev

    def run(self, with_cur=False, current=None, table=None, lengths=None, stream=None, q=None, **kw):
        import torch
        from loop_aware_quantized_b200 import paged_decode
        q = self.q if q is None else q
        lse = torch.full(q.shape[:-1], 7.0, device=self.dev)
        status = ints([0], self.dev)
        cur = self.cur if with_cur else (None, None)
        out = paged_decode(self.cells, q, self.kp, self.vp,
                           ints(self.table if table is None else table, self.dev),
                           ints(self.lengths if lengths is None else lengths, self.dev),
                           meta=self.meta, cur_k=cur[0], cur_v=cur[1], current=current, lse=lse,
                           status=status, stream=stream, **kw)
        torch.cuda.synchronize()
        return out, lse, int(status)

    def check(self, with_cur=False, current=None, table=None, lengths=None, status=0, **kw):
        import torch
        out, lse, st = self.run(with_cur, current, table, lengths, **kw)
        assert st == status
        table = self.table if table is None else table
        lengths = self.lengths if lengths is None else lengths
        cur = tuple(host(x).astype(np.float64) for x in self.cur) if with_cur else None
        meta = None if self.meta is None else host(self.meta)
        ref = R.decode(self.cells, host(self.q), host(self.kp), host(self.vp), meta, table, lengths,
                       self.ps, cur=cur, current=current, sm_scale=kw.get("sm_scale"))
        half = torch.finfo(out.dtype).eps / 2
        n = max(1, int(np.max(lengths)))
        tol, tol_lse = R.bounds(ref[0], ref[2], ref[3], n, half)
        got, got_lse = host(out).astype(np.float64), host(lse).astype(np.float64)
        assert np.isfinite(got).all()
        empty = np.isneginf(ref[1])
        assert np.array_equal(np.isneginf(got_lse), empty) and not got[empty].any()
        worst = (np.abs(got - ref[0]) / tol).max()
        worst_lse = (np.abs(got_lse - ref[1])[~empty] / tol_lse[~empty]).max() if (~empty).any() else 0
        assert worst <= 1 and worst_lse <= 1, (worst, worst_lse)
        return out, lse


EDGES = [0, 1, 2, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 129, 200, 511, 513]


@pytest.mark.parametrize("fmt", ["bf16", "fp16", "q8"])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("group", [1, 4, 8, 16])
def test_decode_lengths(dev, fmt, dim, group):
    Case(dev, fmt, EDGES, heads=2, group=group, dim=dim, seed=group).check()


@pytest.mark.parametrize("group", [2, 3, 5, 7, 9, 15])
def test_decode_odd_groups(dev, group):
    for fmt in ("bf16", "q8"):
        Case(dev, fmt, [40, 7, 300], heads=3, group=group, dim=64, seed=group).check()


@pytest.mark.parametrize("ps", [1, 5, 16, 24, 100, 1024])
@pytest.mark.parametrize("fmt", ["fp16", "q8"])
def test_decode_page_sizes(dev, ps, fmt):
    Case(dev, fmt, [1, 999, 1024, 47, 2048, 2047], heads=1, group=2, dim=128, ps=ps, seed=ps).check()


@pytest.mark.parametrize("fmt", ["bf16", "fp16", "q8"])
@pytest.mark.parametrize("group", [1, 8])
def test_decode_long_requests_are_split(dev, fmt, group):
    Case(dev, fmt, [70001], heads=1, group=group, dim=128, ps=64, seed=3, scale=2.0).check()
    Case(dev, fmt, [9000, 1, 30000], heads=2, group=group, dim=64, ps=16, seed=4, scale=2.0).check()


def test_decode_many_short_requests(dev):
    rng = np.random.default_rng(0)
    Case(dev, "bf16", rng.integers(0, 40, 1500), heads=2, group=2, dim=64, seed=5).check()
    Case(dev, "q8", rng.integers(0, 3, 4096), heads=1, group=1, dim=64, seed=6).check()


@pytest.mark.parametrize("fmt", ["bf16", "fp16", "q8"])
def test_decode_current_tokens(dev, fmt):
    # cells that share pool cell 1 with their own newest token, beside one that reads its own pages
    c = Case(dev, fmt, EDGES, heads=2, group=2, dim=128, cells=(1, 0, 1, 1), seed=7)
    c.check(with_cur=True)
    c.check(with_cur=True, current=[True, False, False, True])
    c.check()


def test_decode_many_cells_of_one_pool_cell(dev):
    # listed cells that read the same tokens, more query rows than one pass over the pages takes
    for fmt, group, times in (("bf16", 1, 37), ("q8", 3, 11), ("fp16", 16, 3)):
        cells = [1, 0] * (times // 2) + [1]
        c = Case(dev, fmt, [33, 0, 700, 1], heads=2, group=group, dim=64, ps=24, cells=cells, seed=18)
        c.check()
        c.check(with_cur=True, current=[i % 3 > 0 for i in range(len(cells))])


def test_decode_rising_maximum(dev):
    # every tile's scores above the last one's, by little and by much
    import torch
    for fmt, step in (("bf16", 0.1), ("bf16", 3.0), ("fp16", 0.1), ("fp16", 3.0), ("bf16", -3.0)):
        c = Case(dev, fmt, [1500], heads=1, group=2, dim=64, ps=16, seed=19)
        c.q[:] = 0.25
        ramp = torch.arange(1500, device=dev) // 16 * step
        page = torch.tensor(c.table[0, :94], device=dev)
        flat = torch.zeros(94 * 16, device=dev)
        flat[:1500] = ramp
        c.kp[0, page, 0] = flat.reshape(94, 16, 1).to(c.kp.dtype)
        c.check()


def test_decode_scale_and_sharp_scores(dev):
    c = Case(dev, "bf16", [300, 5000], heads=2, group=2, dim=64, seed=8, scale=6.0)
    c.check(sm_scale=0.5)
    c.check(sm_scale=0.01)


def test_decode_bad_pages_are_left_out_and_flagged(dev):
    for fmt in ("bf16", "q8"):
        c = Case(dev, fmt, [100, 64, 33, 0], heads=2, group=2, seed=9)
        t = c.table.copy()
        t[0, 2], t[1, :4], t[2, 2] = -1, c.shape[1], 2 ** 31 - 1
        c.check(table=t, status=R.BAD_PAGE)      # request 1 has no page left: zeros, -infinity


def test_decode_bad_lengths_count_as_zero(dev):
    c = Case(dev, "bf16", [100, 64, 33, 20], heads=1, seed=10)
    width = c.table.shape[1]
    n = np.array([100, -1, width * c.ps + 1, 20])
    ref = n.copy()
    ref[1] = ref[2] = 0
    out, lse, st = c.run(lengths=n)
    assert st == R.BAD_LENGTH
    out2, lse2 = c.check(lengths=ref)
    assert (out == out2).all() and (lse == lse2).all()


def test_decode_infinite_scores_and_values(dev):
    # a token whose score is -infinity has no weight; only such tokens: nothing; NaN and
    # +infinity reach the outputs of their own request and head only
    c = Case(dev, "bf16", [20, 20, 20, 20], heads=2, dim=64, seed=11)
    c.q[:] = 1.0
    page = c.table[:, 0]
    c.kp[0, page[0], 0, 3] = float("-inf")
    c.kp[0, page[1], :] = float("-inf")
    c.kp[0, c.table[1, 1], :] = float("-inf")
    c.kp[0, page[2], 1, 2] = float("nan")
    c.vp[0, page[3], 0, 1, 5] = float("inf")
    out, lse, st = c.run()
    o, e = host(out), host(lse)
    assert np.isfinite(o[0, 0]).all() and np.isfinite(e[0, 0]).all()
    assert not o[0, 1].any() and np.isneginf(e[0, 1]).all()
    assert np.isfinite(o[0, 2, 0]).all() and np.isnan(o[0, 2, 1]).all()
    assert np.isposinf(o[0, 3, 0, 5]) and np.isfinite(np.delete(o[0, 3, 0], 5)).all()
    assert np.isfinite(o[0, 3, 1]).all()


def test_decode_fp16_large_values_and_tiny_weights(dev):
    # values at fp16's end, weights of a long even context far below fp16's smallest normal
    c = Case(dev, "fp16", [40000], heads=1, dim=64, ps=64, seed=12, scale=0.01)
    c.vp.copy_(c.vp.nan_to_num(0, 0, 0).clamp(-3, 3) * 20000)
    c.check()


def test_decode_q8_wide_scales(dev):
    # scales from 1e-12 to 1e12 within one request's values
    c = Case(dev, "q8", [600], heads=1, group=2, dim=128, seed=13)
    f = 10.0 ** np.random.default_rng(0).integers(-12, 13, c.shape[:4])
    import torch
    c.meta[..., 2:] *= torch.tensor(f, device=dev, dtype=torch.float32)[..., None]
    out, _, _ = c.run()
    ref = R.decode(c.cells, host(c.q), host(c.kp), host(c.vp), host(c.meta), c.table, c.lengths, c.ps)
    tol, _ = R.bounds(ref[0], ref[2], ref[3], 600, 2.0 ** -8)
    assert (np.abs(host(out) - ref[0]) <= tol).all()


def test_decode_is_deterministic_and_leaves_inputs(dev):
    c = Case(dev, "bf16", [3000, 17, 0, 900], heads=4, group=4, dim=128, seed=14)
    before = [as_bytes(x) for x in (c.kp, c.vp, c.q)]
    a, b = c.run(), c.run()
    assert (a[0] == b[0]).all() and (a[1] == b[1]).all()
    assert all(np.array_equal(x, as_bytes(y)) for x, y in zip(before, (c.kp, c.vp, c.q)))


def test_decode_reads_strided_vectors(dev):
    import torch
    c = Case(dev, "bf16", [100, 5, 64], heads=2, group=2, dim=64, cells=(0, 0), seed=15)
    fused = torch.empty((c.batch, 2, 8, c.dim), dtype=torch.bfloat16, device=dev)  # [batch, cells, q|k|v]
    fused[:, :, :4] = c.q.transpose(0, 1)
    fused[:, :, 4:6], fused[:, :, 6:] = c.cur[0].transpose(0, 1), c.cur[1].transpose(0, 1)
    want = c.run(with_cur=True)
    c.cur = tuple(fused[:, :, a:a + 2].transpose(0, 1) for a in (4, 6))
    got = c.run(with_cur=True, q=fused[:, :, :4].transpose(0, 1))
    assert (got[0] == want[0]).all() and (got[1] == want[1]).all()


def test_decode_reads_broadcast_vectors(dev):
    # one query row, one current token for every cell and request: strides of zero
    import torch
    c = Case(dev, "fp16", [70, 0, 33], heads=2, group=2, dim=64, cells=(0, 0, 0), seed=21)
    c.q = c.q[:1, :1].expand(3, 3, 4, 64)
    c.cur = tuple(x[:1, :, :1].expand(3, 3, 2, 64) for x in c.cur)
    got = c.run(with_cur=True, out=torch.empty((3, 3, 4, 64), dtype=torch.float16, device=dev))
    c.q, c.cur = c.q.contiguous(), tuple(x.contiguous() for x in c.cur)
    want = c.check(with_cur=True)
    assert (got[0] == want[0]).all() and (got[1] == want[1]).all()


def test_decode_of_empty_requests_only(dev):
    for fmt in ("bf16", "q8"):
        c = Case(dev, fmt, [0] * 70, heads=3, group=5, dim=128, cells=(0, 1), seed=22)
        c.check()
        c.check(with_cur=True)


def test_decode_on_another_stream(dev):
    import torch
    c = Case(dev, "bf16", [2000, 300], heads=2, group=2, dim=128, seed=16)
    want = c.run()
    s = torch.cuda.Stream(dev)
    s.wait_stream(torch.cuda.current_stream())
    got = c.run(stream=s)
    assert (got[0] == want[0]).all() and (got[1] == want[1]).all()


@pytest.mark.parametrize("captured", [False, True])
def test_calls_one_after_another_see_each_others_results(dev, captured):
    # kernels are set up while their predecessors run: long in-place maps and releases, appends and
    # decodes back to back, torch's kernels between them, against the same calls one at a time
    import torch
    from loop_aware_quantized_b200 import page_map, page_release, paged_append, paged_decode
    rng = np.random.default_rng(4)
    B, ps, width, rows, heads, dim = 300, 4, 40, 6000, 2, 64
    n_pages = B * width
    new = [np.where(rng.random(B) < 0.7, rng.integers(0, 25, B), 0) for _ in range(4)]
    g = torch.Generator(device=dev).manual_seed(0)
    rand = lambda *sh: torch.randn(sh, generator=g, device=dev).to(torch.bfloat16)  # noqa: E731
    k, v, q = rand(1, rows, heads, dim), rand(1, rows, heads, dim), rand(1, B, heads, dim)
    adds = [ints(x, dev) for x in new]

    def state():
        z = lambda n: ints(np.zeros(n), dev)  # noqa: E731
        return dict(len=z(B), table=ints(np.full((B, width), -1), dev), free=ints(rng2.permutation(n_pages), dev),
                    count=ints([n_pages], dev), slots=z(rows), starts=z(B + 1), cut=z(B), status=z(1),
                    kp=torch.zeros((1, n_pages, heads, ps, dim), dtype=torch.bfloat16, device=dev),
                    vp=torch.zeros((1, n_pages, heads, ps, dim), dtype=torch.bfloat16, device=dev),
                    outs=[torch.zeros_like(q) for _ in adds])

    def run(s, between=lambda: None):
        for i, add in enumerate(adds):
            page_map(s["len"], add, s["table"], s["free"], s["count"], ps, s["slots"], s["starts"], status=s["status"])
            between()
            paged_append([0], k, v, s["slots"], s["kp"], s["vp"], status=s["status"])
            between()
            paged_decode([0], q, s["kp"], s["vp"], s["table"], s["len"], out=s["outs"][i], status=s["status"])
            between()
            torch.div(s["len"], 2, rounding_mode="floor", out=s["cut"])
            page_release(s["len"], s["cut"], s["table"], s["free"], s["count"], ps, status=s["status"])
            between()
            page_release(s["len"], s["cut"], s["table"], s["free"], s["count"], ps, status=s["status"])
            between()

    rng2 = np.random.default_rng(5)
    want = state()
    run(want, torch.cuda.synchronize)
    for _ in range(10):
        rng2 = np.random.default_rng(5)
        got = state()
        if captured:
            side = torch.cuda.Stream(dev)
            side.wait_stream(torch.cuda.current_stream())
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph, stream=side):
                run(got)
            graph.replay()
        else:
            run(got)
        torch.cuda.synchronize()
        for name in ("len", "table", "free", "count", "slots", "starts", "status", "kp", "vp"):
            assert (got[name] == want[name]).all(), name
        assert all((a == b).all() for a, b in zip(got["outs"], want["outs"]))
    assert int(want["status"]) == 0 and sum((o != 0).any() for o in want["outs"]) == 4


def test_every_way_of_calling_gives_the_same(dev):
    # the short way (current stream) and the long one (a stream given, a tensor subclass, cells as
    # a tuple or range), lists and arrays of cells, outputs given or made
    import torch
    from loop_aware_quantized_b200 import paged_append, paged_decode

    class Other(torch.Tensor):
        pass

    c = Case(dev, "q8", [40, 0, 130], heads=2, group=2, dim=64, cells=(1, 0, 1), seed=20)
    t, n = ints(c.table, dev), ints(c.lengths, dev)
    args = (c.kp, c.vp, t, n)
    kw = dict(meta=c.meta, cur_k=c.cur[0], cur_v=c.cur[1])
    flags = [True, False, True]
    want = paged_decode([1, 0, 1], c.q, *args, **kw, current=np.array(flags))
    calls = [dict(cells=x, **kw, current=f) for x, f in (
        ((1, 0, 1), flags), (np.array([1, 0, 1]), np.array(flags)), (np.array([1, 0, 1], np.int32), flags),
        (np.array([1, 0, 1], np.int16), np.array(flags, np.uint8)), ([np.int64(1), 0, 1], tuple(flags)),
        (np.array([1, 5, 0, 5, 1])[::2], np.array(flags)))]
    calls += [dict(cells=[1, 0, 1], **kw, current=flags, stream=torch.cuda.current_stream()),
              dict(cells=[1, 0, 1], **{**kw, "cur_k": c.cur[0].as_subclass(Other)}, current=flags)]
    for call in calls:
        out = torch.full_like(c.q, 5)
        assert paged_decode(q=c.q, k_pages=c.kp, v_pages=c.vp, table=t, lengths=n, out=out, **call) is out
        assert (out == want).all()
        assert (paged_decode(q=c.q, k_pages=c.kp, v_pages=c.vp, table=t, lengths=n, **call) == want).all()
    slots = ints([3, -1, 40], dev)
    pools = []
    for cells, stream in (([1, -1, 0], None), ((1, -1, 0), None), (np.array([1, -1, 0]), torch.cuda.current_stream())):
        pool = [x.clone() for x in (c.kp, c.vp, c.meta)]
        paged_append(cells, c.cur[0], c.cur[1], slots, pool[0], pool[1], meta=pool[2], stream=stream)
        pools.append([as_bytes(x) for x in pool])
    assert all(np.array_equal(x, y) for p in pools[1:] for x, y in zip(p, pools[0]))
    assert not np.array_equal(pools[0][0], as_bytes(c.kp))


def test_calls_at_once_on_two_streams(dev):
    # each call has a workspace of its own
    import torch
    from loop_aware_quantized_b200 import paged_decode
    cases = [Case(dev, "bf16", [20000 + i], heads=2, group=4, dim=128, ps=64, seed=i) for i in range(2)]
    want = [c.run()[0] for c in cases]
    args = [(c.cells, c.q, c.kp, c.vp, ints(c.table, dev), ints(c.lengths, dev)) for c in cases]
    streams = [torch.cuda.Stream(dev) for _ in cases]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(20):
        for i in range(2):
            got[i].append(paged_decode(*args[i], stream=streams[i]))
    torch.cuda.synchronize()
    for i in range(2):
        assert all((g == want[i]).all() for g in got[i])


def test_pages_far_into_a_large_pool(dev):
    # byte offsets past 2^32: the same tokens in the last pages of a 5 GB pool and in a small one
    import torch
    from loop_aware_quantized_b200 import paged_append, paged_decode
    heads, ps, dim, few = 16, 64, 128, 6
    n_pages = 5 * (1 << 30) // (heads * ps * dim * 2)
    lengths, width = ints([130, 64, 100], dev), 3
    near = np.array([[5, 0, 2], [1, -1, -1], [4, 3, -1]])
    far = np.where(near >= 0, n_pages - few + near, -1)
    tables = [ints(near, dev), ints(far, dev)]
    g = torch.Generator(device=dev).manual_seed(3)
    k, v = (torch.randn((1, few * ps, heads, dim), generator=g, device=dev).to(torch.bfloat16) for _ in range(2))
    q = torch.randn((1, 3, 2 * heads, dim), generator=g, device=dev).to(torch.bfloat16)
    outs = []
    for pages, first, table in ((few, 0, tables[0]), (n_pages, n_pages - few, tables[1])):
        kp, vp = (torch.empty((1, pages, heads, ps, dim), dtype=torch.bfloat16, device=dev) for _ in range(2))
        paged_append([0], k, v, ints(np.arange(few * ps) + first * ps, dev), kp, vp)
        outs.append(paged_decode([0], q, kp, vp, table, lengths))
        assert (kp[0, first:].transpose(1, 2).reshape(-1, heads, dim) == k[0]).all()
        del kp, vp
    assert width == 3 and (outs[0] == outs[1]).all() and (outs[0] != 0).any()


def test_longest_request(dev):
    # 2^22 tokens: equal scores give the log of their number and the values' mean
    import math
    import torch
    from loop_aware_quantized_b200 import paged_decode
    n, ps = 1 << 22, 1024
    kp = torch.zeros((1, n // ps, 1, ps, 64), dtype=torch.bfloat16, device=dev)
    vp = torch.full_like(kp, 1.5)
    vp[:, ::2] = -0.5
    table = ints(np.random.default_rng(0).permutation(n // ps)[None], dev)
    lse = torch.zeros((1, 1, 3), device=dev)
    out = paged_decode([0], torch.ones((1, 1, 3, 64), dtype=torch.bfloat16, device=dev), kp, vp, table,
                       ints([n], dev), lse=lse)
    # a warp's sum is exact (whole numbers below 2^24), so are the joined ones
    assert (out == 0.5).all() and (lse - math.log(n)).abs().max() <= 2.0 ** -20 * math.log(n)


def test_two_captured_decodes_have_workspaces_of_their_own(dev):
    # two graphs replayed at once on two streams
    import torch
    from loop_aware_quantized_b200 import paged_decode
    cases = [Case(dev, "bf16", [30000 + i, 10], heads=2, group=4, dim=128, ps=64, seed=30 + i) for i in range(2)]
    want = [c.run()[0] for c in cases]
    args = [(c.cells, c.q, c.kp, c.vp, ints(c.table, dev), ints(c.lengths, dev)) for c in cases]
    outs, graphs, streams = [torch.zeros_like(c.q) for c in cases], [], [torch.cuda.Stream(dev) for _ in cases]
    torch.cuda.synchronize()
    for a, out in zip(args, outs):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            paged_decode(*a, out=out)
            paged_decode(*a, out=out)
        graphs.append(graph)
    for _ in range(30):
        for graph, stream in zip(graphs, streams):
            with torch.cuda.stream(stream):
                graph.replay()
    torch.cuda.synchronize()
    assert all((o == w).all() for o, w in zip(outs, want))


def test_refusals_on_the_device(dev):
    import torch
    from loop_aware_quantized_b200 import paged_append, paged_decode
    from loop_aware_quantized_b200.loopkv import LoopKVError
    c = Case(dev, "bf16", [10, 20], heads=2, group=2, dim=64, seed=17)
    t, n = ints(c.table, dev), ints(c.lengths, dev)
    good = dict(cells=[0], q=c.q, k_pages=c.kp, v_pages=c.vp, table=t, lengths=n)
    wide = torch.zeros((1, 2, 4, 68), dtype=torch.bfloat16, device=dev)
    for bad in (dict(q=c.q.half()), dict(q=c.q[..., :32]), dict(q=c.q[:, :1]), dict(q=c.q[:, :, :3]),
                dict(q=wide[..., 2:66]), dict(q=wide[..., :64]), dict(v_pages=c.vp.half()),
                dict(v_pages=c.vp[:, :1]), dict(table=t.long()), dict(table=t.t()),
                dict(lengths=n[:1]), dict(lengths=n.cpu()), dict(cells=[1]), dict(cells=[]),
                dict(cur_k=c.cur[0]), dict(current=[True]), dict(meta=torch.zeros(1, device=dev)),
                dict(out=torch.zeros_like(c.q, dtype=torch.float32)),
                dict(lse=torch.zeros(3, device=dev)), dict(sm_scale=float("nan"))):
        with pytest.raises(LoopKVError) as e:
            paged_decode(**{**good, **bad})
        assert e.value.status == 1, bad
    s = ints([1, 2], dev)
    for bad in (dict(cells=[0, 0]), dict(k=c.cur[0].float()), dict(slots=s.long()), dict(slots=s[:1]),
                dict(cells=[-2])):
        with pytest.raises(LoopKVError) as e:
            paged_append(**{**dict(cells=[0], k=c.cur[0], v=c.cur[1], slots=s, k_pages=c.kp,
                                   v_pages=c.vp), **bad})
        assert e.value.status == 1, bad


# ------------------------------------------------------------ used together

class Served:
    """A PagedCache and a contiguous host copy of everything it was given."""

    def __init__(self, dev, dtype, shared, batch=5, heads=2, group=2, dim=64, n_pages=40, ps=16,
                 max_pages=8, seed=0):
        import torch
        from loop_aware_quantized_b200 import PagedCache
        self.cache = PagedCache(3, 2, heads, dim, n_pages, ps, batch, max_pages, shared=shared,
                                dtype=dtype, device=dev)
        self.g = torch.Generator(device=dev).manual_seed(seed)
        self.dev, self.batch, self.heads, self.group, self.dim = dev, batch, heads, group, dim
        self.vec = torch.float16 if dtype == torch.float16 else torch.bfloat16
        self.tokens = [[] for _ in range(batch)]        # per request: (k, v) [cells, heads, dim]

    def randn(self, *shape):
        import torch
        return torch.randn(shape, generator=self.g, device=self.dev).to(self.vec)

    def values(self, x):
        """What pages hold of x (fp64)."""
        if self.cache.meta is None:
            return x.astype(np.float64)
        code, scale, zero = R.quantize(x)
        return code * scale[..., None].astype(np.float64) + zero[..., None].astype(np.float64)

    def expected(self, cells, q, step):
        """fp64 outputs of the requests in ``step`` and their magnitudes."""
        c = self.cache
        out, wm = np.zeros(q.shape), np.zeros(q.shape)
        sm = np.zeros(q.shape[:-1])
        for i, cell in enumerate(cells):
            src = (c.n_loops - 1) * c.n_layers + cell % c.n_layers if c.shared[cell] else cell
            for b in step:
                k, v = (np.stack([self.values(t[a][src]) for t in self.tokens[b]], 1) for a in (0, 1))
                if c.shared[cell]:
                    k[:, -1], v[:, -1] = self.tokens[b][-1][0][cell], self.tokens[b][-1][1][cell]
                for h in range(self.heads):
                    qs = q[i, b, h * self.group:(h + 1) * self.group].astype(np.float64)
                    s = qs @ k[h].T * self.dim ** -0.5
                    p = np.exp(s - s.max(-1, keepdims=True))
                    p /= p.sum(-1, keepdims=True)
                    sl = (i, b, slice(h * self.group, (h + 1) * self.group))
                    out[sl], wm[sl] = p @ v[h], p @ np.abs(v[h])
                    sm[sl] = (np.abs(qs) @ np.abs(k[h]).T * self.dim ** -0.5).max(-1)
        return out, wm, sm


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "q8"])
@pytest.mark.parametrize("captured", [False, True])
def test_serving_run(dev, dtype, captured):
    # prompts, decode steps in serving order (captured once and replayed), a pausing request, a
    # rollback, an ended request whose pages another takes
    import torch
    from loop_aware_quantized_b200 import steps
    s = Served(dev, torch_dtype(dtype), shared=[0, 1, 3])
    c, B = s.cache, s.batch
    cells = np.arange(c.n_cells)

    def prompts(new):
        rows = int(sum(new)) + 3
        slots = ints(np.zeros(rows), dev)
        c.grow(ints(new, dev), slots)
        k, v = s.randn(c.n_cells, rows, s.heads, s.dim), s.randn(c.n_cells, rows, s.heads, s.dim)
        c.append(cells, k, v, slots)
        kh, vh, r = host(k), host(v), 0
        for b, n in enumerate(new):
            for _ in range(n):
                s.tokens[b].append((kh[:, r], vh[:, r]))
                r += 1

    phases = steps.phases(c.n_loops, c.n_layers)
    shape = lambda p, h: (len(p), B, h, s.dim)  # noqa: E731
    q = [s.randn(*shape(p, s.heads * s.group)) for p in phases]
    k, v = ([s.randn(*shape(p, s.heads)) for p in phases] for _ in range(2))
    out = [torch.zeros_like(x) for x in q]
    ones, slots = ints(np.ones(B), dev), ints(np.zeros(B), dev)
    graph = None
    if captured:
        side = torch.cuda.Stream(dev)
        side.wait_stream(torch.cuda.current_stream())
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            steps.paged_decode_step(c, phases, ones, slots, q, k, v, out)

    def step(active):
        for x in (*q, *k, *v):
            x.copy_(s.randn(*x.shape))
        ones.copy_(ints([int(b in active) for b in range(B)], dev))
        if graph is not None:
            graph.replay()
        else:
            steps.paged_decode_step(c, phases, ones, slots, q, k, v, out)
        torch.cuda.synchronize()
        kh, vh = (np.concatenate([host(x) for x in y]) for y in (k, v))
        for b in active:
            s.tokens[b].append((kh[:, b], vh[:, b]))
        for p, qq, oo in zip(phases, q, out):
            ref, wm, sm = s.expected(p, host(qq), active)
            if dtype == "q8":      # codes up to 255 steps around the zero point: |x| + range
                wm, sm = 4 * wm + 4, 4 * sm + 4
            tol, _ = R.bounds(ref, wm, sm, 200, torch.finfo(s.vec).eps / 2)
            assert (np.abs(host(oo) - ref)[:, active] <= tol[:, active]).all()
        assert host(c.lengths).tolist() == [len(t) for t in s.tokens]

    prompts([20, 0, 33, 1, 64])
    for _ in range(3):
        step([0, 2, 3, 4])
    step([0, 2, 4])                      # request 3 pauses
    prompts([0, 17, 0, 0, 0])
    for _ in range(18):                  # every request crosses a page's end
        step([0, 1, 2, 3, 4])
    c.cut(ints([max(0, len(t) - d) for t, d in zip(s.tokens, (3, 0, 40, 0, 200))], dev))
    for b, d in enumerate((3, 0, 40, 0, 200)):
        s.tokens[b] = s.tokens[b][:max(0, len(s.tokens[b]) - d)]
    held = sum(-(-len(t) // 16) for t in s.tokens)
    assert int(c.free_count) == 40 - held
    step([0, 1, 2, 3])
    prompts([0, 0, 0, 30, 90])
    step([0, 1, 2, 3, 4])
    c.check()
    table, n = host(c.table), host(c.lengths)
    pages = [table[b, j] for b in range(B) for j in range(-(-n[b] // 16))]
    free = host(c.free)[:int(c.free_count)].tolist()
    assert sorted(pages + free) == list(range(40))       # no page lost, none twice


def test_cache_reports_refused_requests(dev):
    from loop_aware_quantized_b200.loopkv import LoopKVError
    import torch
    s = Served(dev, torch.bfloat16, shared=[], n_pages=3)
    slots = ints(np.zeros(200), dev)
    s.cache.grow(ints([20, 30, 40, 0, 0], dev), slots)
    with pytest.raises(LoopKVError) as e:
        s.cache.check()
    assert e.value.status == 3                           # LOOPKV_ERR_CAPACITY
    assert host(s.cache.lengths).tolist() == [20, 0, 0, 0, 0] and int(s.cache.free_count) == 1
    s.cache.check()                                      # cleared


def test_paged_cells_agree_with_a_plan(dev):
    # bf16 and SHARE cells of a plan and of a paged cache, given the same tokens and queries
    import torch
    from loop_aware_quantized_b200 import LOOPKV_BF16, LOOPKV_SHARE, PagedCache, Plan, steps
    L, N, H, D, B, n = 2, 2, 3, 128, 4, 70
    kinds = np.full(L * N, LOOPKV_BF16, np.uint8)
    kinds[1] = LOOPKV_SHARE
    plan = Plan(L, N, H, D, np.full(B, 128, np.int32), kinds, tau=0.0)
    cache = PagedCache(L, N, H, D, 32, 16, B, 8, shared=[1], device=dev)
    slots, grow = ints(np.zeros(B * n), dev), ints(np.full(B, n), dev)
    g = torch.Generator(device=dev).manual_seed(1)
    rand = lambda *sh: torch.randn(sh, generator=g, device=dev).to(torch.bfloat16)  # noqa: E731
    cells = np.arange(L * N)
    k, v = rand(L * N, B, H, n, D), rand(L * N, B, H, n, D)
    plan.append(cells, k, v)
    cache.grow(grow, slots)
    flat = lambda x: x.permute(0, 1, 3, 2, 4).reshape(L * N, B * n, H, D)  # noqa: E731
    cache.append(cells, flat(k), flat(v), slots)
    phases = steps.phases(L, N)
    q = [rand(len(p), B, H, D) for p in phases]
    kn, vn = ([rand(len(p), B, H, D) for p in phases] for _ in range(2))
    a = [torch.zeros(x.shape, dtype=torch.float32, device=dev) for x in q]
    b = [torch.zeros_like(x) for x in q]
    steps.decode_step(plan, phases, q, [x[:, :, :, None] for x in kn], [x[:, :, :, None] for x in vn], a)
    steps.paged_decode_step(cache, phases, ints(np.ones(B), dev), ints(np.zeros(B), dev), q, kn, vn, b)
    torch.cuda.synchronize()
    plan.check()
    cache.check()
    for x, y in zip(a, b):
        # both are within 1e-4 of the exact value (weights to 2^-16 of values below 5); the paged
        # one is rounded to bf16
        assert (x - y.float()).abs().max() <= 2e-4 + 2.0 ** -8 * float(x.abs().max())
    plan.close()
