"""Plain 64-bit forms of the paged cells' operators, one request at a time, and
the bounds their GPU results are held to.  No code of the library is used."""

import math

import numpy as np

BAD_LENGTH, NO_TABLE, NO_ROWS, NO_PAGES, BAD_PAGE, BAD_SLOT = 1, 2, 4, 8, 16, 32


def page_map(lengths, new, table, free, count, ps, rows):
    """(table, slots, starts, lengths_out, count_out, status) of the definition."""
    table = table.copy()
    batch, width = table.shape
    n_pages = free.size
    slots = np.full(rows, -1, np.int64)
    starts = np.zeros(batch + 1, np.int64)
    out = lengths.astype(np.int64).copy()
    status, asked = 0, 0
    if not 0 <= count <= n_pages:
        status, count = BAD_LENGTH, 0
    have = count
    for b in range(batch):
        n, a = int(lengths[b]), int(new[b])
        starts[b + 1] = starts[b] + max(a, 0)
        if n < 0 or a < 0:
            status |= BAD_LENGTH
            continue
        if n + a > width * ps:
            status |= NO_TABLE
            continue
        if starts[b + 1] > rows:
            status |= NO_ROWS
            continue
        held, need = -(-n // ps), -(-(n + a) // ps) - -(-n // ps)
        asked += need
        if need and asked > have:
            status |= NO_PAGES
            continue
        for j in range(held, held + need):
            page = int(free[count - 1])
            count -= 1
            table[b, j] = page if 0 <= page < n_pages else -1
        for i in range(a):
            page, off = int(table[b, (n + i) // ps]), (n + i) % ps
            if 0 <= page < n_pages:
                slots[starts[b] + i] = page * ps + off
            else:
                status |= BAD_PAGE
        out[b] = n + a
    return table, slots, np.minimum(starts, 2 ** 31 - 1), out, count, status


def page_release(lengths, new, table, free, count, ps):
    """(free, lengths_out, count_out, status)."""
    free = free.copy()
    batch, width = table.shape
    out = lengths.astype(np.int64).copy()
    status, room, asked = 0, free.size - count, 0
    if not 0 <= count <= free.size:
        status, count, room = BAD_LENGTH, 0, 0      # nothing is pushed, no page is offered
    for b in range(batch):
        n, a = int(lengths[b]), int(new[b])
        if a < 0 or a > n or n > width * ps:
            status |= BAD_LENGTH
            continue
        first, last = -(-a // ps), -(-n // ps)
        asked += last - first
        if last > first and asked > room:
            status |= NO_PAGES
            continue
        for j in range(first, last):
            page = int(table[b, j])
            if not 0 <= page < free.size:
                status |= BAD_PAGE
                page = -1
            free[count] = page
            count += 1
        out[b] = a
    return free, out, count, status


def quantize(x):
    """8-bit codes, scale and zero point over the last axis, in fp32 steps."""
    x = x.astype(np.float32)
    low, high = x.min(-1, keepdims=True), x.max(-1, keepdims=True)
    scale = ((high - low) / np.float32(255)).astype(np.float32)
    with np.errstate(divide="ignore", invalid="ignore"):
        code = np.where(scale > 0, np.rint(((x - low) / scale).astype(np.float32)), 0)
    zero = np.where(low == 0, np.float32(0), low)
    return np.clip(code, 0, 255).astype(np.uint8), scale[..., 0], zero[..., 0]


def stored(pages, meta, part):
    """fp64 values of a page tensor, and the sum of the magnitudes they are made of."""
    x = pages.astype(np.float64)
    if meta is None:
        return x, np.abs(x)
    scale, zero = (meta[..., part + i, None].astype(np.float64) for i in (0, 1))
    return scale * x + zero, np.abs(scale * x) + np.abs(zero)


def decode(cells, q, k_pages, v_pages, meta, table, lengths, ps, cur=None, current=None,
           sm_scale=None):
    """(out, lse, weight magnitude, score magnitude) in fp64; pages as numpy
    arrays, tokens of pages outside the pool left out.  The last two are what
    rounding errors are relative to: sum_t p_t |v_t| and max_t scale sum_d
    |q_d k_td|."""
    nc, batch, heads_q, dim = q.shape
    heads, n_pages = k_pages.shape[2], k_pages.shape[1]
    g = heads_q // heads
    scale = dim ** -0.5 if sm_scale is None else sm_scale
    q = q.astype(np.float64)
    out = np.zeros(q.shape)
    lse = np.full(q.shape[:-1], -math.inf)
    wmag, smag = np.zeros(q.shape), np.zeros(q.shape[:-1])
    for i, c in enumerate(cells):
        cur_here = cur is not None and (current is None or current[i])
        for b in range(batch):
            n = int(lengths[b])
            if n <= 0 or n > table.shape[1] * ps:
                continue
            pos = np.arange(n - 1 if cur_here else n)
            page = table[b, pos // ps]
            ok = (page >= 0) & (page < n_pages)
            page, off = page[ok], pos[ok] % ps
            for h in range(heads):
                mk = mv = None
                if meta is not None:
                    mk = mv = meta[c, page, h, off]
                k, ka = stored(k_pages[c, page, h, off], mk, 0)
                v, va = stored(v_pages[c, page, h, off], mv, 2)
                if cur_here:
                    k, v = (np.concatenate([x, y[i, b, h][None].astype(np.float64)])
                            for x, y in ((k, cur[0]), (v, cur[1])))
                    ka, va = (np.concatenate([x, np.abs(y[i, b, h][None].astype(np.float64))])
                              for x, y in ((ka, cur[0]), (va, cur[1])))
                if not len(k):
                    continue
                qs = q[i, b, h * g:(h + 1) * g]
                s = scale * qs @ k.T
                top = s.max(-1, keepdims=True)
                p = np.exp(s - top)
                total = p.sum(-1, keepdims=True)
                out[i, b, h * g:(h + 1) * g] = p @ v / total
                lse[i, b, h * g:(h + 1) * g] = (top + np.log(total))[:, 0]
                wmag[i, b, h * g:(h + 1) * g] = p @ va / total
                smag[i, b, h * g:(h + 1) * g] = (scale * np.abs(qs) @ ka.T).max(-1)
    return out, lse, wmag, smag


def bounds(out, wmag, smag, n, half):
    """(|error| allowed for out, for lse).  A score is a sum of D products in
    fp32 with at most a unit in the last place (2^-23) lost per 16-wide step
    and per factor it meets, 16 of them at most: 2^-19 of the magnitudes, and as
    much again for the 2^-24 roundings of scale and exponent argument: 2^-18.
    A weight is that far off relatively, twice over with the sum it is
    divided by, plus 2^-16 for its pair of 16-bit floats (bf16: 2^-8 twice)
    and 2^-21 for the exponential; n / 16 steps over the tokens lose 2^-23 each.
    The output is rounded once to its type, by half a step (``half``)."""
    score = 2.0 ** -18 * smag
    w = 2 * score + 2.0 ** -16 + 2.0 ** -20 + n * 2.0 ** -27
    tol = w[..., None] * wmag
    return tol + half * (np.abs(out) + tol) + 2.0 ** -24, score + 2.0 ** -20 + n * 2.0 ** -27
