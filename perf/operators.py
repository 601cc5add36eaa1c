"""Measured cases of the operators that read and copy the KV pool's rows.

  selected  attention of each verify query's heads over its k selected rows,
            read where their location vector says (tail ring, optional page,
            hot cache), split over k and joined
  history   attention of new tokens over a source's whole history (or a
            drafter's window): tail ring and paged history, split over its
            length and joined
  fork      a request's pages, tail ring, hot cache and host rows copied into
            another request slot (and the slot's previous request freed)
  recycle   the request in the lowest page slots is freed, the remaining pages
            are moved down into the holes, the freed request is forked anew

A row of the pool holds `kv_heads` key heads and value heads.  In the latent
layout (kv == 0) one key of `key` elements is shared by all query heads and
the value is its first `value` elements; otherwise the row is [kv][key]
keys followed by [kv][value] values.
"""
import math
import random

import torch

own = False

PAGE = 64
NO_LOC = 0xFFFFFFFF
DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16}


# ------------------------------------------------------------------- cases

def _selected(name, requests, queries, topk, heads, *, key=576, value=512, kv=0, hot=4096,
              tail=256, pages=512, lost=0.0, overlap=0.8, dtype="bf16"):
    return dict(name=name, op="selected", requests=requests, queries=queries, topk=topk,
                heads=heads, key=key, value=value, kv=kv, hot=hot, tail=tail, pages=pages,
                lost=lost, overlap=overlap, dtype=dtype)


def _history(name, requests, queries, rows, heads, *, key=576, value=512, kv=0, tail=256,
             window=False, ragged=0.0, dtype="bf16"):
    return dict(name=name, op="history", requests=requests, queries=queries, rows=rows,
                heads=heads, key=key, value=value, kv=kv, tail=tail, window=window,
                ragged=ragged, dtype=dtype)


def _pages(name, op, sources, rows, *, hot=4096, tail=256, cold=4):
    return dict(name=name, op=op, sources=sources, rows=rows, hot=hot, tail=tail, cold=cold)


def listed():
    return [
        # one request's single new token on the smallest pool (4096-row
        # history, 256 selected rows): launch latency counts
        _selected("selected_one", 1, 1, 256, 16, hot=512, tail=64, pages=64),
        # one layer of decoding at concurrency 8: 2048 selected rows each,
        # a 16-head shard of the model
        _selected("selected_decode8", 8, 1, 2048, 16),
        # one layer of speculative verification at concurrency 64: blocks of
        # 8 queries that share 80 % of their rows
        _selected("selected_verify64", 64, 8, 2048, 16),
        # the same layer unsharded, all 128 heads on this GPU, concurrency 16
        _selected("selected_heads128", 16, 8, 2048, 128),
        # odd sizes: grouped heads, f16 rows, entries without a row
        _selected("selected_grouped", 24, 3, 777, 40, key=128, value=128, kv=8,
                  hot=2000, tail=100, pages=100, lost=0.07, dtype="f16"),
        # a drafter's window at concurrency 128: the ring of its last 512 rows
        _history("window_draft128", 128, 1, 900, 32, tail=512, window=True),
        # a dense layer's new token over 32K-row histories, concurrency 8
        _history("history_32k", 8, 1, 32768, 16),
        # one request's new token over a 500K-row history: split over length
        _history("history_500k", 1, 1, 512000, 16),
        # a verify block of 4 on grouped heads, histories of ragged lengths
        _history("history_grouped", 12, 4, 9000, 32, key=128, value=128, kv=4, ragged=0.9),
        # a fork of the smallest request (4096 rows, one source)
        _pages("fork_small", "fork", 1, 4096, hot=512, tail=64),
        # a fork of a 32K-row request with four sources
        _pages("fork_32k", "fork", 4, 32768),
        # a 100K-row request finishes, the pool is compacted, a new one forked
        _pages("recycle_100k", "recycle", 1, 102400),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["selected", "selected", "history", "history", "fork", "recycle"])
    if op in ("selected", "history"):
        grouped = rng.random() < 0.35
        kv = rng.choice([1, 2, 4, 8]) if grouped else 0
        heads = kv * rng.randint(1, 8) if grouped else _log(rng, 1, 128)
        dims = dict(key=rng.choice([64, 96, 128]), value=rng.choice([64, 128]), kv=kv) \
            if grouped else dict(key=576, value=512, kv=0)
        dtype = rng.choice(["bf16", "bf16", "f16"])
    if op == "selected":
        queries = rng.choice([1, 1, 2, 4, 8])
        topk = _log(rng, 64, 2048)
        requests = max(1, min(64, int(_log(rng, 1, 1024) / queries), (16 * 128) // max(1, heads)))
        case = _selected(None, requests, queries, topk, heads, hot=rng.randint(512, 4096),
                         tail=rng.randint(32, 256), pages=rng.randint(64, 512),
                         lost=rng.choice([0.0, 0.0, 0.05]), overlap=rng.choice([0.0, 0.5, 0.8]),
                         dtype=dtype, **dims)
    elif op == "history":
        queries = rng.choice([1, 1, 4, 8])
        window = rng.random() < 0.3
        rows = _log(rng, 64, 2048 if window else 200000)
        rows = min(rows, 30_000_000 // (heads * queries))  # no more products than listed ones
        elems = kv * (dims["key"] + dims["value"]) if kv else 576
        requests = max(1, min(_log(rng, 1, 128), 290_000 * 576 // (elems * rows),
                              30_000_000 // (rows * heads * queries)))
        case = _history(None, requests, queries, rows, heads, window=window,
                        tail=rng.randint(1 + rows // 4, rows) if window else rng.randint(64, 400),
                        ragged=rng.choice([0.0, 0.5, 0.95]), dtype=dtype, **dims)
    else:
        sources = rng.choice([1, 2, 4])
        case = _pages(None, op, sources, _log(rng, 640, 100000 // sources),
                      hot=rng.randint(256, 4096), tail=rng.randint(16, 256),
                      cold=rng.randint(1, 4))
    del case["name"]
    return case


# ------------------------------------------------------------------ inputs

def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _row_elems(c):
    return c["kv"] * (c["key"] + c["value"]) if c["kv"] else c["key"]


def _randn(shape, dtype, g):
    out = torch.empty(shape, dtype=dtype, device=DEV)
    return out.normal_(generator=g)


def _lengths(c, seed):
    """Length of each request's history: `rows`, or down to (1 - ragged) of it."""
    r = random.Random(seed)
    lo = max(1, int(c["rows"] * (1 - c["ragged"])))
    return [c["rows"] if not c["ragged"] else r.randint(lo, c["rows"]) for _ in range(c["requests"])]


def _prep_selected(c, seed):
    g, dt, E = _gen(seed), TYPES[c["dtype"]], _row_elems(c)
    R, Q, k = c["requests"], c["queries"], c["topk"]
    # the tiers (tail, pages, hot) side by side, each 256-byte aligned
    rows = [R * c["tail"], R * c["pages"] * PAGE, R * c["hot"]]
    first, n = [], 0
    for m in rows:
        first.append(n)
        n += -(-m // 16) * 16
    arena = _randn((n, E), dt, g)
    # every request's rows: its tail ring, its pages (scattered slots), its hot slots
    slots = torch.randperm(R * c["pages"], generator=g, device=DEV).view(R, -1, 1)
    r = torch.arange(R, device=DEV).view(R, 1)
    at = lambda m: r * m + torch.arange(m, device=DEV)  # noqa: E731
    pages = (slots * PAGE + torch.arange(PAGE, device=DEV)).view(R, -1)
    every = torch.cat([at(c["tail"]), pages + (1 << 30), at(c["hot"]) + (2 << 30)], 1)
    core = int(c["overlap"] * k) if Q > 1 else 0
    order = torch.rand((R, every.shape[1]), generator=g, device=DEV).argsort(1)
    pick = torch.cat([order[:, None, :core].expand(R, Q, core),
                      order[:, core:core + Q * (k - core)].reshape(R, Q, k - core)], 2)
    loc = every.gather(1, pick.reshape(R, -1)).view(R, Q, k)
    loc[torch.rand(loc.shape, generator=g, device=DEV) < c["lost"]] = NO_LOC
    return dict(case=c, arena=arena, tiers=list(zip(first, rows)),
                first=torch.tensor(first + [0], device=DEV),
                loc=loc.to(torch.int32).contiguous(), q=_randn((R, Q, c["heads"], c["key"]), dt, g),
                out=torch.empty((R, Q, c["heads"], c["value"]), dtype=dt, device=DEV),
                lse=torch.empty((R, Q, c["heads"]), device=DEV))


def _prep_history(c, seed):
    g, dt = _gen(seed), TYPES[c["dtype"]]
    R, Q, lens = c["requests"], c["queries"], _lengths(c, seed)
    rows = _randn((R, c["rows"], _row_elems(c)), dt, g)
    return dict(case=c, lens=lens, npages=[0 if c["window"] else n // PAGE for n in lens],
                history=rows, q=_randn((R, Q, c["heads"], c["key"]), dt, g),
                out=torch.empty((R, Q, c["heads"], c["value"]), dtype=dt, device=DEV),
                lse=torch.empty((R, Q, c["heads"]), device=DEV))


def _prep_pages(c, seed):
    """Requests 0 (the parent), 1 and 2 (its copies, in that slot order), each
    with `sources` histories; the oldest `cold` pages of each live in host
    memory, and their rows are in the hot cache."""
    g, S, n = _gen(seed), c["sources"], c["rows"]
    m = min(c["cold"] * PAGE, c["hot"])
    return dict(case=c, turn=0, rows=_randn((S, n, 576), torch.bfloat16, g),
                picked=torch.arange(m, dtype=torch.int32, device=DEV).repeat(S, 1),
                host=torch.empty((3, S, n, 576), dtype=torch.int16, pin_memory=True))


def prepare(case, seed):
    s = {"selected": _prep_selected, "history": _prep_history, "fork": _prep_pages,
         "recycle": _prep_pages}[case["op"]](case, seed)
    # what a program keeps between calls: the pool with its arenas, descriptors
    # and workspace, or the same layout in plain tensors
    if own:
        keep = {"selected": _own_selected, "history": _own_history}.get(case["op"], _own_pages)
    else:
        keep = {"selected": _plain_selected, "history": _plain_history}.get(case["op"], _plain_pages)
    keep(s)
    torch.cuda.synchronize()
    for name in ("history", "rows"):
        s.pop(name, None)
    return s


# ------------------------------------------------------- the framework's own

def _heads(c):
    """The row layout's arguments of dhs.make_attend."""
    kv = c["kv"]
    return dict(heads=c["heads"], kv_heads=max(1, kv), key_elems=c["key"],
                value_elems=c["value"], value_offset=kv * c["key"],
                scale=c["key"] ** -0.5, dtype=c["dtype"])


def _own_attend(s, items):
    from hierarchical_sparse_kv_dhs_gb300 import dhs
    s["at"], s["keep"] = dhs.make_attend(items, **_heads(s["case"]))
    s["work"] = torch.zeros(max(256, s["pool"].attend_bytes(s["at"])), dtype=torch.uint8, device=DEV)
    s["at"].work_dev, s["at"].work_bytes = s["work"].data_ptr(), s["work"].numel()


def _own_selected(s):
    from hierarchical_sparse_kv_dhs_gb300 import dhs
    c = s["case"]
    rb = _row_elems(c) * 2
    flat = s["arena"].view(torch.uint8).view(-1)
    tail, opt, hot = [flat[f * rb:(f + m) * rb] for f, m in s["tiers"]]
    s["pool"] = dhs.Pool(max_requests=c["requests"], sources=1, row_bytes=rb, page_rows=PAGE,
                         tail_rows=c["tail"], hot_rows=c["hot"], max_queries=c["queries"],
                         max_topk=c["topk"], max_rows_per_request=(c["pages"] + 8) * PAGE,
                         optional_pages=c["requests"] * c["pages"],
                         arenas=(hot, tail, opt))
    items = [dhs.attend_item(queries=c["queries"], topk=c["topk"], q=s["q"][r], loc=s["loc"][r],
                             out=s["out"][r], lse=s["lse"][r]) for r in range(c["requests"])]
    _own_attend(s, items)


def _own_history(s):
    from hierarchical_sparse_kv_dhs_gb300 import dhs
    c, lens = s["case"], s["lens"]
    rb = _row_elems(c) * 2
    s["pool"] = dhs.Pool(max_requests=c["requests"], sources=1, row_bytes=rb, page_rows=PAGE,
                         tail_rows=c["tail"], hot_rows=16, max_queries=c["queries"], max_topk=16,
                         max_rows_per_request=c["rows"], optional_pages=sum(s["npages"]))
    if not c["window"]:
        s["host"] = torch.empty((c["requests"], c["rows"] * rb), dtype=torch.uint8, pin_memory=True)
    for r, n in enumerate(lens):
        if c["window"]:
            m = min(n, c["tail"])
            dhs.check(s["pool"].admit_window(r, 0, s["history"][r, n - m:].data_ptr(), n))
        else:
            dhs.check(s["pool"].admit_device(r, 0, s["history"][r].data_ptr(),
                                             s["host"][r].data_ptr(), n)[0])
    dhs.check(s["pool"].flush())
    items = [dhs.attend_item(req=r, queries=c["queries"], flags=dhs.DHS_ATTEND_HISTORY, q=s["q"][r],
                             out=s["out"][r], lse=s["lse"][r]) for r in range(c["requests"])]
    _own_attend(s, items)


def _own_pages(s):
    from hierarchical_sparse_kv_dhs_gb300 import dhs
    c, host = s["case"], s["host"]
    S, n, m = c["sources"], c["rows"], s["picked"].shape[1]
    P = n // PAGE
    pool = s["pool"] = dhs.Pool(max_requests=3, sources=S, row_bytes=1152, page_rows=PAGE,
                                tail_rows=c["tail"], hot_rows=c["hot"], max_queries=1, max_topk=m,
                                max_rows_per_request=n, optional_pages=3 * S * (P - c["cold"]))
    for b in pool.buffers[:3]:
        b.zero_()
    mask = [0] * c["cold"] + [1] * (P - c["cold"])
    loc, items = torch.empty_like(s["picked"]), []
    for i in range(S):
        dhs.check(pool.admit_device(0, i, s["rows"][i].data_ptr(), host[0, i].data_ptr(), n, mask)[0])
        it = dhs.dhs_item()
        it.src, it.queries, it.topk = i, 1, m
        it.sel_dev, it.loc_dev = s["picked"][i].data_ptr(), loc[i].data_ptr()
        items.append(it)
    st, keep = dhs.make_step(1, items)
    dhs.check(pool.resolve(st))
    s["hosts"] = [[host[r, i].data_ptr() for i in range(S)] for r in range(3)]
    for r in (1, 2):
        dhs.check(pool.fork(0, r, s["hosts"][r])[0])
    s["hot"], s["tail"], s["opt"] = [b.view(torch.int16) for b in pool.buffers[:3]]
    dhs.check(pool.status()[0])


def _run_own(s):
    from hierarchical_sparse_kv_dhs_gb300 import dhs
    op, pool = s["case"]["op"], s["pool"]
    if op in ("selected", "history"):
        dhs.check(pool.attend(s["at"]), "dhs_attend")
        return [s["out"], s["lse"]]
    child = 1 + s["turn"]
    dhs.check(pool.release(child), "dhs_release")
    if op == "recycle":  # the other copy's pages move down into the freed slots
        dhs.check(pool.compact(pool.used())[0], "dhs_compact")
        dhs.check(pool.compact(pool.cfg.optional_pages)[0], "dhs_compact")
        s["turn"] ^= 1
    dhs.check(pool.fork(0, child, s["hosts"][child])[0], "dhs_fork")
    return [s["hot"], s["tail"], s["opt"]] + _outside(s, child)


def _outside(s, r):
    """Request r's host rows that no resident page holds."""
    c, host = s["case"], s["host"]
    return [host[r, :, :c["cold"] * PAGE], host[r, :, c["rows"] // PAGE * PAGE:]]


# ------------------------------------------------------------- plain forms

def _attend(q, k, v, keep, scale):
    """softmax(scale q k^T) v over the kept rows: q [B, C, d], k [B, n, d],
    v [B, n, e], keep [B, C or 1, n]; a row with nothing kept gives zeros and
    a log-sum of -inf."""
    s = torch.matmul(q, k.transpose(1, 2)) * scale
    s = s.masked_fill(~keep, float("-inf"))
    m = s.amax(2, keepdim=True)
    p = torch.exp(s - m.masked_fill(m == float("-inf"), 0))
    z = p.sum(2, keepdim=True)
    o = torch.matmul(p, v) / z.masked_fill(z == 0, 1)
    return o, (m + torch.log(z)).squeeze(2)


def _split(c, rows):
    """Keys and values [kv, ..., n, d] of rows [..., n, E]."""
    if not c["kv"]:
        return rows[None], rows[None, ..., :c["value"]]
    G, n = c["kv"], c["kv"] * c["key"]
    k = rows[..., :n].unflatten(-1, (G, c["key"])).movedim(-2, 0)
    v = rows[..., n:].unflatten(-1, (G, c["value"])).movedim(-2, 0)
    return k, v


def _plain_selected(s):
    pass  # the arena, its tiers' first rows and the locations are the plain layout


def _plain_run_selected(s):
    c = s["case"]
    R, Q, H = s["q"].shape[:3]
    outs = []
    for r in range(0, R, 16):  # the selected rows of 16 requests at a time
        loc = s["loc"][r:r + 16].long() & 0xFFFFFFFF
        keep = loc < 0xC0000000
        at = torch.where(keep, s["first"][loc >> 30] + (loc & 0x3FFFFFFF), 0)
        b = len(loc)
        rows = s["arena"][at].float().view(b * Q, c["topk"], -1)
        outs.append(_grouped(c, s["q"][r:r + 16].float().view(b * Q, 1, H, -1), rows,
                             keep.view(b * Q, 1, -1)))
    return _joined(outs, s)


def _grouped(c, q, rows, keep):
    """Attention of q [b, Q, H, d] over rows [b, n, E] by groups of heads; keep [b, Q, n]."""
    b, Q, H = q.shape[:3]
    G, n = max(1, c["kv"]), rows.shape[1]
    k, v = _split(c, rows)
    q = q.view(b, Q, G, H // G, -1).permute(2, 0, 1, 3, 4).reshape(G * b, Q * H // G, -1)
    keep = keep[None, :, :, None].expand(G, b, Q, H // G, n).reshape(G * b, Q * H // G, n)
    o, lse = _attend(q, k.reshape(G * b, n, -1), v.reshape(G * b, n, -1), keep, c["key"] ** -0.5)
    o = o.view(G, b, Q, H // G, -1).permute(1, 2, 0, 3, 4).reshape(b * Q, H, -1)
    return o, lse.view(G, b, Q, H // G).permute(1, 2, 0, 3).reshape(b * Q, H)


def _joined(outs, s):
    o, lse = (torch.cat(x) for x in zip(*outs))
    return [o.view(s["out"].shape).to(s["out"].dtype), lse.view(s["lse"].shape)]


def _plain_history(s):
    """Pages in one arena with the tail rings behind them, and the page table."""
    c, E = s["case"], s["history"].shape[-1]
    R, T, lens = c["requests"], c["tail"], s["lens"]
    total, first = sum(s["npages"]), 0
    s["arena"] = torch.zeros((total * PAGE + R * T, E), dtype=s["q"].dtype, device=DEV)
    s["table"] = torch.zeros((R, max(1, max(s["npages"]))), dtype=torch.int64, device=DEV)
    s["ring"] = torch.arange(R, device=DEV) * T + total * PAGE
    for r, n in enumerate(lens):
        m = s["npages"][r]
        s["table"][r, :m] = torch.arange(first, first + m, device=DEV)
        s["arena"][first * PAGE:(first + m) * PAGE] = s["history"][r, :m * PAGE]
        first += m
        last = torch.arange(max(0, n - T), n, device=DEV)
        s["arena"][s["ring"][r] + last % T] = s["history"][r, last]
    s["len"] = torch.tensor(lens, device=DEV)


def _plain_run_history(s):
    c = s["case"]
    R, Q, T = c["requests"], c["queries"], c["tail"]
    lo = max(0, min(s["lens"]) - T) if c["window"] else 0
    pos = torch.arange(lo, max(s["lens"]), device=DEV)
    outs = []
    per = max(1, 600_000_000 // (len(pos) * s["arena"].shape[1]))
    for r in range(0, R, per):  # as many histories at a time as fit in 2.4 GB
        n, tab = s["len"][r:r + per, None], s["table"][r:r + per]
        page = tab[:, (pos // PAGE).clamp(max=tab.shape[1] - 1)] * PAGE + pos % PAGE
        at = torch.where(pos >= n - T, s["ring"][r:r + per, None] + pos % T, page)
        # query i of the block is the row L - Q + i: it sees itself and what precedes it
        end = n - (Q - 1) + torch.arange(Q, device=DEV)
        keep = pos < end[..., None]
        if c["window"]:
            keep = keep & (pos >= n - T)[:, None]
        outs.append(_grouped(c, s["q"][r:r + per].float(), s["arena"][at].float(), keep))
    return _joined(outs, s)


def _plain_pages(s):
    """The pool's arenas as tensors, the parent and both copies in place."""
    c, rows, host = s["case"], s["rows"].view(torch.int16), s["host"]
    S, n, B, T, m = c["sources"], c["rows"], c["hot"], c["tail"], s["picked"].shape[1]
    P, cold = n // PAGE, c["cold"]
    warm = P - cold
    zeros = lambda *shape: torch.zeros(shape, dtype=torch.int16, device=DEV)  # noqa: E731
    s["hot"], s["tail"], s["opt"] = zeros(3, S, B, 576), zeros(3, S, T, 576), zeros(3 * S * warm, PAGE, 576)
    s["tags"] = torch.full((3, S, B), -1, dtype=torch.int32, device=DEV)
    s["stamps"] = torch.zeros((3, S, B), dtype=torch.int32, device=DEV)
    s["map"] = torch.full((3, S, P), -1, dtype=torch.int64, device=DEV)
    s["map"][0, :, cold:] = torch.arange(S * warm, device=DEV).view(S, warm)
    s["opt"][:S * warm] = rows[:, cold * PAGE:P * PAGE].reshape(S * warm, PAGE, 576)
    last = torch.arange(max(0, n - T), n, device=DEV)
    s["tail"][0, :, last % T] = rows[:, last]
    s["hot"][0, :, :m], s["tags"][0, :, :m], s["stamps"][0, :, :m] = rows[:, :m], s["picked"], 1
    host[0, :, :cold * PAGE] = rows[:, :cold * PAGE].cpu()
    host[0, :, P * PAGE:] = rows[:, P * PAGE:].cpu()
    for r in (1, 2):
        _plain_fork(s, r, r * S * warm)


def _plain_fork(s, child, slot):
    n = len(s["opt"]) // 3
    for name in ("hot", "tail", "tags", "stamps"):
        s[name][child] = s[name][0]
    s["map"][child] = torch.where(s["map"][0] >= 0, s["map"][0] + slot, -1)
    s["opt"][slot:slot + n] = s["opt"][:n]
    for to, of in zip(_outside(s, child), _outside(s, 0)):
        to.copy_(of)


def _plain_run_pages(s):
    n, child = len(s["opt"]) // 3, 1 + s["turn"]
    s["tags"][child], s["stamps"][child], s["map"][child] = -1, 0, -1
    slot = child * n
    if s["case"]["op"] == "recycle":  # the other copy lies in the upper third
        other = s["map"][3 - child]
        s["opt"][n:2 * n] = s["opt"][2 * n:]
        s["map"][3 - child] = torch.where(other >= 0, other - n, -1)
        slot = 2 * n
        s["turn"] ^= 1
    _plain_fork(s, child, slot)
    return [s["hot"].view(-1), s["tail"].view(-1), s["opt"].view(-1)] + _outside(s, child)


def run(state):
    if own:
        return _run_own(state)
    plain = {"selected": _plain_run_selected, "history": _plain_run_history}
    return plain.get(state["case"]["op"], _plain_run_pages)(state)


# ------------------------------------------------------------ work and truth

def work(case):
    c = case
    if c["op"] in ("fork", "recycle"):
        S, P = c["sources"], c["rows"] // PAGE
        pages = S * (P - c["cold"]) * PAGE
        rows = pages + S * (c["tail"] + min(c["cold"] * PAGE, c["hot"]) + c["cold"] * PAGE + c["rows"] % PAGE)
        if c["op"] == "recycle":
            rows += pages  # moved down
        return {"bytes": 2 * (rows * 1152 + S * (8 * c["hot"] + 4 * P)), "flops": 0}
    heads = c["requests"] * c["queries"] * c["heads"]
    io = heads * (2 * (c["key"] + c["value"]) + 4)
    if c["op"] == "selected":
        R, Q, k = c["requests"], c["queries"], c["topk"]
        core = int(c["overlap"] * k) if Q > 1 else 0
        rows = R * (core + Q * (k - core)) * (1 - c["lost"])
        pairs = heads * k * (1 - c["lost"])
        io += 4 * R * Q * k
    else:
        rows = c["requests"] * min(c["rows"], c["tail"] if c["window"] else c["rows"]) * (1 - c["ragged"] / 2)
        pairs = rows * c["queries"] * c["heads"]
    return {"bytes": rows * _row_elems(c) * 2 + io, "flops": 2 * pairs * (c["key"] + c["value"])}


def exact(case, seed):
    c = case
    if c["op"] in ("fork", "recycle"):
        return None  # copies: no computed numbers
    s = (_prep_selected if c["op"] == "selected" else _prep_history)(c, seed)
    R, Q, H = s["q"].shape[:3]
    out = torch.zeros(s["out"].shape, dtype=torch.float64, device=DEV)
    lse = torch.full(s["lse"].shape, float("-inf"), dtype=torch.float64, device=DEV)
    share = H // max(1, c["kv"])
    for r in range(R):
        for i in range(Q):
            if c["op"] == "selected":
                loc = s["loc"][r, i].long() & 0xFFFFFFFF
                loc = loc[loc != NO_LOC]
                rows = s["arena"][s["first"][loc >> 30] + (loc & 0x3FFFFFFF)]
            else:
                n = s["lens"][r]
                rows = s["history"][r, max(0, n - c["tail"]) if c["window"] else 0:max(0, n - Q + 1 + i)]
            if not len(rows):
                continue
            for h in range(0, H, share):
                at = h // share
                lo = at * c["key"]
                key = rows[:, lo:lo + c["key"]].double()
                lo = c["kv"] * c["key"] + at * c["value"]
                value = rows[:, lo:lo + c["value"]].double()
                x = s["q"][r, i, h:h + share].double() @ key.T / math.sqrt(c["key"])
                lse[r, i, h:h + share] = torch.logsumexp(x, 1)
                out[r, i, h:h + share] = torch.softmax(x, 1) @ value
    return [out, lse]
