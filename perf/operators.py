"""The paged key-value cache's operators as they are measured.

A server keeps the cache of every (loop, layer) cell in pages.  A step asks for room for its new tokens
(``page_map``: block tables, slot map), writes their keys and values into it (``paged_append``), lets every
request's newest token attend over its pages (``paged_decode``), and gives pages back when requests end or
are cut (``page_release``).  Cases are measured one operator at a time.

Layouts: pages [cells, pages, KV heads, page size, head dim]; table [requests, pages of the longest]; slots
[rows] with slot = page * page size + offset.  Pages behind a request's length hold whatever was there before:
here NaN and infinities among it.
"""

import math

import torch

own = False  # run() makes the framework's calls where true, the plain form where not

DEV = "cuda"
BF16, F16, Q8 = "bf16", "fp16", "q8"


def listed():
    return [
        # One decode step of 32 requests at 16K context: every call of a serving loop starts with this one.
        {"name": "map step", "op": "map", "batch": 32, "ctx": 16384, "page": 64, "rows": 32, "mode": "step", "short": False},
        # A batch of prompts admitted at once, small pages: a million rows of slot map.
        {"name": "map prompts", "op": "map", "batch": 256, "ctx": 0, "page": 16, "rows": 1 << 20, "mode": "prompts", "short": False},
        # A few requests of a small batch ended; the others go on.
        {"name": "release some", "op": "release", "batch": 33, "ctx": 4096, "page": 64, "ended": 0.2},
        # A whole wave of requests ends, small pages.
        {"name": "release wave", "op": "release", "batch": 1024, "ctx": 16384, "page": 16, "ended": 0.9},
        # One token of 32 requests for the 72 cells of three loops over 24 layers (16 heads of 128), one call.
        {"name": "append step", "op": "append", "format": BF16, "cells": 72, "rows": 32, "heads": 16, "dim": 128, "page": 64, "fill": 1.0},
        # A prompt chunk of one cell, padded behind its last row.
        {"name": "append prompt", "op": "append", "format": F16, "cells": 1, "rows": 40001, "heads": 16, "dim": 128, "page": 16, "fill": 0.9},
        # The same into 8-bit pages: quantized on the way.
        {"name": "append prompt q8", "op": "append", "format": Q8, "cells": 2, "rows": 16384, "heads": 16, "dim": 128, "page": 32, "fill": 1.0},
        # One layer, one request: the smallest call of interactive use.
        {"name": "decode one", "op": "decode", "format": BF16, "cells": 1, "batch": 1, "heads": 16, "group": 1, "dim": 128, "page": 64, "total": 4113, "cap": 5120, "even": True, "current": False},
        # One layer at the batched 16K workload: 32 requests of 16384 tokens, 4.3 GB of pages.
        {"name": "decode batched", "op": "decode", "format": BF16, "cells": 1, "batch": 32, "heads": 16, "group": 1, "dim": 128, "page": 64, "total": 32 * 16384, "cap": 16384, "even": True, "current": False},
        # Ragged batch with padding rows, query groups of 4, narrow heads, small pages.
        {"name": "decode ragged", "op": "decode", "format": F16, "cells": 2, "batch": 67, "heads": 8, "group": 4, "dim": 64, "page": 16, "total": 120001, "cap": 8192, "even": False, "current": False},
        # Two long documents, one KV head with 8 queries each in 8-bit pages: the length has to be split.
        {"name": "decode long q8", "op": "decode", "format": Q8, "cells": 1, "batch": 2, "heads": 2, "group": 8, "dim": 128, "page": 32, "total": 200003, "cap": 131072, "even": False, "current": False},
        # Cells of three loops that reuse the final loop's pages, with their own newest token.
        {"name": "decode shared", "op": "decode", "format": BF16, "cells": 3, "batch": 8, "heads": 16, "group": 2, "dim": 128, "page": 64, "total": 8 * 4096, "cap": 8192, "even": False, "current": True},
    ]


def _log(rng, low, high):
    return min(high, max(low, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def draw(rng):
    op = rng.choice(["map", "release", "append", "decode", "decode"])
    page = rng.choice([16, 16, 24, 32, 64, 64, 128])
    if op == "map":
        mode = rng.choice(["step", "prompts", "chunk"])
        batch = _log(rng, 1, 1024)
        rows = batch if mode == "step" else _log(rng, 4 * batch, min(1 << 20, batch << 16))
        return {"op": op, "batch": batch, "ctx": 0 if mode == "prompts" else _log(rng, 64, 16384), "page": page, "rows": rows,
                "mode": mode, "short": rng.random() < 0.25}
    if op == "release":
        return {"op": op, "batch": _log(rng, 1, 1024), "ctx": _log(rng, 64, 16384), "page": page, "ended": rng.choice([0.0, 0.1, 0.5, 1.0])}
    form, dim = rng.choice([BF16, F16, Q8]), rng.choice([64, 128])
    if op == "append":
        cells, heads = _log(rng, 1, 72), rng.choice([1, 2, 4, 5, 8, 16])
        rows = _log(rng, 1, max(1, (1 << 26) // (cells * heads * dim)))
        return {"op": op, "format": form, "cells": cells, "rows": rows, "heads": heads, "dim": dim, "page": page, "fill": rng.choice([0.6, 1.0])}
    cells, heads, batch = _log(rng, 1, 24), rng.choice([1, 2, 4, 5, 8, 16]), _log(rng, 1, 128)
    cap = _log(rng, 32, 131072)
    most = max(1, min(batch * cap // 4, (1 << 28) // (cells * heads * dim)))
    even = rng.random() < 0.3
    return {"op": op, "format": form, "cells": cells, "batch": batch, "heads": heads, "group": rng.choice([1, 1, 2, 3, 4, 7, 8, 16]), "dim": dim,
            "page": page, "total": _log(rng, max(1, most // 64), most), "cap": min(cap, max(32, 4 * most // batch)), "even": even, "current": rng.random() < 0.3}


# ------------------------------------------------------------------- inputs

def _ceil(a, b):
    return (a + b - 1) // b


def _generator(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _lengths(g, batch, total, cap, even):
    """Request lengths that add up to about `total`, none above `cap`; ragged ones have requests without a token."""
    if even:
        n = torch.full((batch,), max(1, min(cap, total // batch)), device=DEV)
        return n.to(torch.int32)
    w = -torch.rand(batch, generator=g, device=DEV, dtype=torch.float64).clamp_min(1e-9).log()
    if batch > 8:
        w[torch.rand(batch, generator=g, device=DEV) < 0.05] = 0
    for _ in range(16):  # what the cap cuts off goes to the others
        w = w.clamp_max(cap)
        w = w * (total / w.sum())
    n = w.clamp_max(cap).floor()
    n[0] = n[0].clamp_min(1)
    return n.to(torch.int32)


def _tables(g, lengths, width, page, n_pages):
    """A block table with pages in random order, and the pages that are left as the free list."""
    batch = lengths.numel()
    order = torch.randperm(n_pages, generator=g, device=DEV).to(torch.int32)
    held = _ceil(lengths.long(), page)
    first = held.cumsum(0) - held
    j = torch.arange(width, device=DEV)
    at = first[:, None] + j
    table = torch.where(j < held[:, None], order[at.clamp_max(n_pages - 1)], torch.full((batch, width), -1, dtype=torch.int32, device=DEV))
    used = int(held.sum())
    free = torch.full((n_pages,), -1, dtype=torch.int32, device=DEV)
    free[: n_pages - used] = order[used:]
    return table.contiguous(), free, torch.tensor([n_pages - used], dtype=torch.int32, device=DEV)


def _int(*shape):
    return torch.zeros(shape, dtype=torch.int32, device=DEV)


def _prepare_map(case, g):
    batch, page, rows, mode = case["batch"], case["page"], case["rows"], case["mode"]
    ctx = torch.rand(batch, generator=g, device=DEV) * 0.5 + 0.5
    lengths = (ctx * case["ctx"]).to(torch.int32)
    if mode == "step":
        new = (torch.rand(batch, generator=g, device=DEV) < 0.97).to(torch.int32)
    else:
        w = -torch.rand(batch, generator=g, device=DEV, dtype=torch.float64).clamp_min(1e-9).log()
        if mode == "chunk":  # most requests decode one token, a few bring a chunk of a prompt
            w = torch.where(torch.rand(batch, generator=g, device=DEV) < 0.8, torch.zeros_like(w), w)
            new = 1 + (w * ((rows - batch) * 0.97 / w.sum().clamp_min(1e-9))).floor().to(torch.int32)
        else:
            new = (w * (rows * 0.97 / w.sum())).floor().to(torch.int32)
    width = _ceil(case["ctx"] + rows, page) if mode != "step" else _ceil(case["ctx"], page) + 1
    width = min(width, _ceil(case["ctx"] + (1 << 17), page))
    n_pages = batch * (_ceil(case["ctx"], page) + 2) + _ceil(rows, page)
    table, free, count = _tables(g, lengths, width, page, n_pages)
    if case["short"]:  # the pool runs dry part of the way through the batch
        need = _ceil(lengths.long() + new, page) - _ceil(lengths.long(), page)
        count = torch.minimum(count, (need.sum() * 0.6).to(torch.int32).reshape(1))
    return {"op": "map", "page": page, "lengths": lengths, "new": new, "table": table, "free": free, "count": count,
            "slots": _int(rows), "starts": _int(batch + 1), "lengths_out": _int(batch), "count_out": _int(1)}


def _prepare_release(case, g):
    batch, page = case["batch"], case["page"]
    lengths = ((torch.rand(batch, generator=g, device=DEV) * 0.9 + 0.1) * case["ctx"]).to(torch.int32)
    width = _ceil(case["ctx"], page)
    n_pages = batch * width + 64
    table, free, count = _tables(g, lengths, width, page, n_pages)
    u = torch.rand(batch, generator=g, device=DEV)
    # ended requests go to zero, a few are cut back (rejected drafts), the rest stays
    cut = (lengths - torch.randint(0, 9, (batch,), generator=g, device=DEV)).clamp_min(0)
    target = torch.where(u < case["ended"], torch.zeros_like(lengths), torch.where(u > 0.95, cut, lengths)).to(torch.int32)
    return {"op": "release", "page": page, "lengths": lengths, "target": target, "table": table, "free": free, "count": count,
            "lengths_out": _int(batch), "count_out": _int(1)}


def _numbers(g, shape, dtype, scale=1.0):
    x = torch.empty(shape, dtype=dtype, device=DEV)
    return x.normal_(0.0, scale, generator=g)


def _pool(g, format, shape):
    """Pages full of earlier tokens: (k, v, meta)."""
    if format != Q8:
        dt = torch.bfloat16 if format == BF16 else torch.float16
        return _numbers(g, shape, dt), _numbers(g, shape, dt), None
    k = torch.randint(0, 256, shape, generator=g, device=DEV, dtype=torch.uint8)
    v = torch.randint(0, 256, shape, generator=g, device=DEV, dtype=torch.uint8)
    meta = torch.rand(shape[:-1] + (4,), generator=g, device=DEV)
    meta[..., 0::2] = meta[..., 0::2] * 0.01 + 0.015  # scales
    meta[..., 1::2] = -128 * meta[..., 0::2] + (meta[..., 1::2] - 0.5)  # zero points
    return k, v, meta


def _prepare_append(case, g):
    cells, rows, heads, dim, page = (case[k] for k in ("cells", "rows", "heads", "dim", "page"))
    dt = torch.float16 if case["format"] == F16 else torch.bfloat16
    n_pages = _ceil(rows, page) + 3
    n_slots = n_pages * page
    slots = torch.randperm(n_pages, generator=g, device=DEV)[torch.arange(rows, device=DEV) // page] * page + torch.arange(rows, device=DEV) % page
    if rows < 4096:  # single tokens of many requests: slots all over the pages
        slots = torch.randperm(n_slots, generator=g, device=DEV)[:rows]
    used = max(1, int(rows * case["fill"]))
    slots[used:] = -1  # rows behind the last sequence
    # per-channel spread of keys, as the framework's synthetic workloads have it
    k = _numbers(g, (cells, rows, heads, dim), dt)
    k *= torch.exp(torch.randn((cells, 1, heads, dim), generator=g, device=DEV)).to(dt)
    v = _numbers(g, (cells, rows, heads, dim), dt)
    kp, vp, meta = _pool(g, case["format"], (cells, n_pages, heads, page, dim))
    return {"op": "append", "page": page, "cells": list(range(cells)), "k": k, "v": v, "slots": slots.to(torch.int32), "kp": kp, "vp": vp, "meta": meta}


def _prepare_decode(case, g):
    cells, batch, heads, group, dim, page = (case[k] for k in ("cells", "batch", "heads", "group", "dim", "page"))
    dt = torch.float16 if case["format"] == F16 else torch.bfloat16
    lengths = _lengths(g, batch, case["total"], case["cap"], case["even"])
    width = _ceil(case["cap"], page)
    n_pages = _ceil(case["total"], page) + batch + 2
    if case["even"]:
        n_pages = batch * _ceil(max(1, min(case["cap"], case["total"] // batch)), page) + 1
    table, _, _ = _tables(g, lengths, width, page, n_pages)
    held = 1 if case["current"] else cells  # cells that share read one stored cell
    kp, vp, meta = _pool(g, case["format"], (held, n_pages, heads, page, dim))
    last = lengths.long() - 1
    tail = torch.zeros((n_pages, page), dtype=torch.bool, device=DEV)  # offsets behind the last token of the last page
    has = last >= 0
    ends = table.gather(1, (last.clamp_min(0) // page)[:, None])[:, 0].long()[has]
    tail[ends] = torch.arange(page, device=DEV) > (last[has] % page)[:, None]
    at = tail.nonzero()
    if meta is None:
        kp[:, at[:, 0], :, at[:, 1]] = float("nan")
        vp[:, at[:, 0], :, at[:, 1]] = float("inf")
    else:
        meta[:, at[:, 0], :, at[:, 1]] = float("nan")
    q = _numbers(g, (cells, batch, heads * group, dim), dt, 3.0)  # scores a few units apart: some tokens matter, most hardly do
    st = {"op": "decode", "page": page, "cells": [0] * cells if case["current"] else list(range(cells)), "q": q, "kp": kp, "vp": vp, "meta": meta, "table": table,
          "lengths": lengths, "group": group, "cur_k": None, "cur_v": None,
          "out": torch.zeros_like(q), "lse": torch.zeros(q.shape[:-1], dtype=torch.float32, device=DEV)}
    if case["current"]:
        st["cur_k"], st["cur_v"] = _numbers(g, (cells, batch, heads, dim), dt), _numbers(g, (cells, batch, heads, dim), dt)
    return st


def prepare(case, seed):
    return {"map": _prepare_map, "release": _prepare_release, "append": _prepare_append, "decode": _prepare_decode}[case["op"]](case, _generator(seed))


# --------------------------------------------------------------- plain forms

def _plain_map(st):
    page, lengths, new, table = st["page"], st["lengths"].long(), st["new"].long(), st["table"]
    batch, width = table.shape
    rows = st["slots"].numel()
    stop = new.cumsum(0)
    starts = stop - new
    held = _ceil(lengths, page)
    ok = (lengths >= 0) & (new >= 0) & (lengths + new <= width * page) & (stop <= rows)
    need = torch.where(ok, _ceil(lengths + new, page) - held, torch.zeros_like(held))
    upto = need.cumsum(0)
    ok = ok & ((need == 0) | (upto <= st["count"]))
    before = upto - need
    need = torch.where(ok, need, torch.zeros_like(need))
    j = torch.arange(width, device=table.device)
    is_new = (j >= held[:, None]) & (j < (held + need)[:, None])
    at = (st["count"].long() - 1 - (before[:, None] + j - held[:, None])).clamp(0, st["free"].numel() - 1)
    table.copy_(torch.where(is_new, st["free"][at], table))
    r = torch.arange(rows, device=table.device)
    b = torch.searchsorted(stop, r, right=True).clamp_max(batch - 1)
    pos = lengths[b] + r - starts[b]
    slot = table[b, (pos // page).clamp(0, width - 1)].long() * page + pos % page
    st["slots"].copy_(torch.where((r < stop[-1]) & ok[b], slot, torch.full_like(slot, -1)))
    st["starts"][1:] = stop
    st["lengths_out"].copy_(torch.where(ok, lengths + new, lengths))
    st["count_out"].copy_(st["count"] - need.sum())
    return st["table"], st["slots"], st["starts"], st["lengths_out"], st["count_out"]


def _plain_release(st):
    page, lengths, target, table = st["page"], st["lengths"].long(), st["target"].long(), st["table"]
    j = torch.arange(table.shape[1], device=table.device)
    gone = (j >= _ceil(target, page)[:, None]) & (j < _ceil(lengths, page)[:, None])
    n = gone.sum()
    flat = gone.reshape(-1)
    at = st["count"].long() + flat.cumsum(0) - 1
    sink = torch.cat([st["free"], st["free"].new_zeros(1)])  # the entries that stay go to the extra place
    sink[torch.where(flat, at, torch.full_like(at, st["free"].numel()))] = table.reshape(-1)
    st["free"].copy_(sink[:-1])
    st["lengths_out"].copy_(target)
    st["count_out"].copy_(st["count"] + n)
    return st["free"], st["lengths_out"], st["count_out"]


def _quantized(x):
    x = x.float()
    low, high = x.amin(-1, keepdim=True), x.amax(-1, keepdim=True)
    scale = (high - low) / torch.full_like(low, 255.0)  # by a tensor: torch divides by a number with its reciprocal
    code = torch.where(scale > 0, ((x - low) / scale).round(), torch.zeros_like(x)).clamp(0, 255)
    return code.to(torch.uint8), scale, low


def _plain_append(st):
    keep = st["slots"] >= 0
    s = st["slots"][keep].long()
    to, off = s // st["page"], s % st["page"]
    k, v = st["k"][:, keep], st["v"][:, keep]
    if st["meta"] is not None:
        (k, ks, kz), (v, vs, vz) = _quantized(k), _quantized(v)
        st["meta"][:, to, :, off] = torch.cat([ks, kz, vs, vz], -1).transpose(0, 1)
    st["kp"][:, to, :, off] = k.transpose(0, 1)
    st["vp"][:, to, :, off] = v.transpose(0, 1)
    # codes are whole numbers and are compared as such; the scales and zero points beside them give their values
    return [st["kp"], st["vp"]] + ([st["meta"]] if st["meta"] is not None else [])


def _plain_decode(st):
    q, table, lengths, group = st["q"].float(), st["table"].long().clamp_min(0), st["lengths"].long(), st["group"]
    cells = torch.tensor(st["cells"], device=q.device) if len(set(st["cells"])) > 1 else st["cells"][:1]
    width, page = table.shape[1], st["page"]
    heads, dim = st["kp"].shape[2], st["kp"].shape[4]
    t = torch.arange(width * page, device=q.device)
    inside = (t < (lengths - (1 if st["cur_k"] is not None else 0))[:, None])[:, None, :, None]  # [batch, 1, tokens, 1]

    def read(pages, part):
        x = pages[cells][:, table].transpose(2, 3).float()  # [cells, batch, heads, pages, page, dim]
        if st["meta"] is not None:
            m = st["meta"][cells][:, table].transpose(2, 3)
            x = m[..., part:part + 1] * x + m[..., part + 1:part + 2]
        return torch.where(inside, x.reshape(x.shape[0], x.shape[1], heads, width * page, dim), torch.zeros((), device=q.device))

    q = q.reshape(q.shape[0], q.shape[1], heads, group, dim)
    s = torch.matmul(q, read(st["kp"], 0).transpose(-1, -2)) / math.sqrt(dim)
    s = torch.where(inside.transpose(-1, -2), s, torch.full((), -math.inf, device=q.device))
    if st["cur_k"] is not None:
        own_s = (q * st["cur_k"].float()[:, :, :, None]).sum(-1, keepdim=True) / math.sqrt(dim)
        s = torch.cat([s, torch.where((lengths > 0)[:, None, None, None], own_s, torch.full_like(own_s, -math.inf))], -1)
    m = s.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, torch.zeros_like(m), m)
    p = (s - m).exp()
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p[..., : width * page], read(st["vp"], 2))
    if st["cur_k"] is not None:
        o = o + p[..., -1:] * st["cur_v"].float()[:, :, :, None]
    o = torch.where(total > 0, o / total.clamp_min(1e-38), torch.zeros_like(o))
    st["out"].copy_(o.reshape(st["out"].shape))
    st["lse"].copy_((m + total.log()).reshape(st["lse"].shape))
    return st["out"], st["lse"]


# ----------------------------------------------------------------------- run

def _own(st):
    import loop_aware_quantized_b200 as lk
    if st["op"] == "map":
        lk.page_map(st["lengths"], st["new"], st["table"], st["free"], st["count"], st["page"], st["slots"], st["starts"],
                    lengths_out=st["lengths_out"], free_count_out=st["count_out"])
        return st["table"], st["slots"], st["starts"], st["lengths_out"], st["count_out"]
    if st["op"] == "release":
        lk.page_release(st["lengths"], st["target"], st["table"], st["free"], st["count"], st["page"],
                        lengths_out=st["lengths_out"], free_count_out=st["count_out"])
        return st["free"], st["lengths_out"], st["count_out"]
    if st["op"] == "append":
        lk.paged_append(st["cells"], st["k"], st["v"], st["slots"], st["kp"], st["vp"], meta=st["meta"])
        return [st["kp"], st["vp"]] + ([st["meta"]] if st["meta"] is not None else [])
    lk.paged_decode(st["cells"], st["q"], st["kp"], st["vp"], st["table"], st["lengths"], meta=st["meta"],
                    cur_k=st["cur_k"], cur_v=st["cur_v"], out=st["out"], lse=st["lse"])
    return st["out"], st["lse"]


def run(state):
    if own:
        return _own(state)
    return {"map": _plain_map, "release": _plain_release, "append": _plain_append, "decode": _plain_decode}[state["op"]](state)


def work(case):
    if case["op"] == "map":
        # lengths in and out, starts, a table entry a request, the free list's and the table's entries of new pages, the slot map
        new_pages = case["rows"] / case["page"]
        return {"bytes": 20 * case["batch"] + 8 * new_pages + 4 * case["rows"], "flops": 0}
    if case["op"] == "release":
        return {"bytes": 12 * case["batch"] + 8 * case["ended"] * case["batch"] * 0.55 * case["ctx"] / case["page"], "flops": 0}
    if case["op"] == "append":
        n = case["cells"] * max(1, int(case["rows"] * case["fill"])) * case["heads"]
        out = 2 * case["dim"] + 16 if case["format"] == Q8 else 4 * case["dim"]
        return {"bytes": n * (4 * case["dim"] + out) + 4 * case["rows"], "flops": 6 * n * case["dim"] if case["format"] == Q8 else 0}
    per = 2 * case["dim"] + 16 if case["format"] == Q8 else 4 * case["dim"]
    total = case["batch"] * max(1, min(case["cap"], case["total"] // case["batch"])) if case["even"] else case["total"]
    read = (1 if case["current"] else case["cells"]) * total * case["heads"] * per
    queries = case["cells"] * case["batch"] * case["heads"] * case["group"]
    return {"bytes": read + queries * (4 * case["dim"] + 4) + 4 * total / case["page"],
            "flops": 4 * case["cells"] * total * case["heads"] * case["group"] * case["dim"]}


# --------------------------------------------------------------------- exact

def _exact_append(case, st):
    """A row at a time into copies of the pages; codes are whole numbers that fp32 defines, so only their scales have a value here."""
    page, slots = st["page"], st["slots"].tolist()
    keep = torch.tensor([i for i, s in enumerate(slots) if s >= 0], device=DEV)
    flat = torch.tensor([s for s in slots if s >= 0], device=DEV)
    if case["format"] == Q8:
        meta = st["meta"].double().permute(0, 1, 3, 2, 4).reshape(case["cells"], -1, case["heads"], 4).clone()
        for part, x in ((0, st["k"]), (2, st["v"])):
            x = x.double()[:, keep]
            low = x.min(-1).values
            meta[:, flat, :, part] = (x.max(-1).values - low) / 255.0
            meta[:, flat, :, part + 1] = low
        return [None, None, meta.reshape(case["cells"], -1, page, case["heads"], 4).permute(0, 1, 3, 2, 4).contiguous()]
    got = []
    for pages, x in ((st["kp"], st["k"]), (st["vp"], st["v"])):
        y = pages.double().permute(0, 1, 3, 2, 4).reshape(case["cells"], -1, case["heads"], case["dim"]).clone()
        y[:, flat] = x.double()[:, keep]
        got.append(y.reshape(case["cells"], -1, page, case["heads"], case["dim"]).permute(0, 1, 3, 2, 4).contiguous())
    return got


def _exact_decode(case, st):
    """One request of one cell at a time: its tokens gathered page by page, a softmax in 64 bits."""
    page, group, dim, heads = st["page"], case["group"], case["dim"], case["heads"]
    out = torch.zeros(st["q"].shape, dtype=torch.float64, device=DEV)
    lse = torch.full(st["lse"].shape, -math.inf, dtype=torch.float64, device=DEV)
    lengths = st["lengths"].tolist()
    for i, c in enumerate(st["cells"]):
        for b, n in enumerate(lengths):
            if n == 0:
                continue
            stored = n - 1 if case["current"] else n
            ids = st["table"][b, : _ceil(stored, page)].long()
            parts = []
            for pages, cur, part in ((st["kp"], st["cur_k"], 0), (st["vp"], st["cur_v"], 2)):
                x = pages[c, ids].double()
                if st["meta"] is not None:
                    m = st["meta"][c, ids].double()
                    x = x * m[..., part, None] + m[..., part + 1, None]
                x = x.transpose(0, 1).reshape(heads, -1, dim)[:, :stored]
                if case["current"]:
                    x = torch.cat([x, cur[i, b].double()[:, None]], 1)
                parts.append(x)
            s = torch.einsum("hgd,htd->hgt", st["q"][i, b].double().reshape(heads, group, dim), parts[0]) * dim ** -0.5
            lse[i, b] = torch.logsumexp(s, -1).reshape(-1)
            out[i, b] = torch.einsum("hgt,htd->hgd", torch.softmax(s, -1), parts[1]).reshape(-1, dim)
    return out, lse


def exact(case, seed):
    if case["op"] in ("map", "release"):
        return None  # whole numbers only
    if case["op"] == "decode" and case["cells"] * case["batch"] > 3000:
        return None
    st = prepare(case, seed)
    return _exact_append(case, st) if case["op"] == "append" else _exact_decode(case, st)
