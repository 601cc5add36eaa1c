"""Measured cases of the operators around rows that the pool holds in 8 bits.

  rotate   rotary positions applied to a step's queries
  append   a verify block's new rows rotated, quantised and appended to a
           drafter's window, and read back in 16 bits
  store    a prompt's rows rotated and quantised into rows of the pool's
           layout, and read back in 16 bits
  read     selected rows, or a source's history, read back in 16 bits
  attend   attention of each query's heads over its selected rows, or of new
           tokens over a source's history, read in 8 bits where they lie

A packed row: [kv][key8] key codes, [kv][value] value codes (none when the
value is the beginning of the key), [kv][wide] elements that stay in 16 bits
(the end of each key head), a 32-bit scale for each key head and each value
head, and padding to 16 bytes.  A code is an e4m3 number; a head's scale is
the smallest power of two that brings its largest element to 448 or below.
"""
import math
import random

import torch

own = False

PAGE = 64
NO_LOC = 0xFFFFFFFF
DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16}
LATENT = dict(kv=1, key=576, wide=64, value=512, shared=True)


def _grouped(kv, key, value, wide=0):
    return dict(kv=kv, key=key, wide=wide, value=value, shared=False)


# ------------------------------------------------------------------- cases

def _rotate(name, tokens, heads, elems, *, offset=0, rotary=None, pairs="half", scaling="plain",
            far=4096, dtype="bf16"):
    return dict(name=name, op="rotate", tokens=tokens, heads=heads, elems=elems, offset=offset,
                rotary=rotary or elems, pairs=pairs, scaling=scaling, far=far, dtype=dtype)


def _write(name, op, requests, tokens, layout, *, rotary, offset, pairs="half", scaling="plain",
           far=4096, window=512, dtype="bf16"):
    return dict(name=name, op=op, requests=requests, tokens=tokens, rotary=rotary, offset=offset,
                pairs=pairs, scaling=scaling, far=far, window=window, dtype=dtype, **layout)


def _located(name, op, requests, queries, topk, heads, layout, *, hot=4096, tail=256, pages=512,
             lost=0.0, overlap=0.8, dtype="bf16"):
    return dict(name=name, op=op, over="located", requests=requests, queries=queries, topk=topk,
                heads=heads, hot=hot, tail=tail, pages=pages, lost=lost, overlap=overlap,
                dtype=dtype, **layout)


def _history(name, op, requests, queries, rows, heads, layout, *, tail=256, ragged=0.0,
             dtype="bf16"):
    return dict(name=name, op=op, over="history", requests=requests, queries=queries, rows=rows,
                heads=heads, tail=tail, ragged=ragged, dtype=dtype, **layout)


def listed():
    return [
        # the queries of one decode step at concurrency 64, blocks of 8: the
        # last 64 of each head's 576 elements turn
        _rotate("rotate_verify64", 512, 16, 576, offset=512, rotary=64, pairs="interleaved"),
        # a prompt's queries in a model whose context was stretched to 1M
        _rotate("rotate_prompt", 8192, 32, 128, scaling="parts", far=1 << 20),
        # a decode step's new rows at concurrency 8: launch latency counts
        _write("append_decode8", "append", 8, 1, LATENT, rotary=64, offset=512, pairs="interleaved"),
        # a prompt of 16K tokens, 8 kv heads whose keys turn whole
        _write("store_prompt", "store", 1, 16384, _grouped(8, 128, 128), rotary=128, offset=0,
               scaling="parts", far=1 << 20),
        # staging for an attention in 16 bits: a verify block's selected rows
        _located("read_verify16", "read", 16, 8, 2048, 16, LATENT),
        # a prefix read back for the next chunk of its prompt, f16, ragged
        _history("read_grouped", "read", 12, 1, 9000, 8, _grouped(4, 96, 64), ragged=0.9,
                 dtype="f16"),
        # one request's single new token, 256 selected rows of the smallest pool
        _located("attend_one", "attend", 1, 1, 256, 16, LATENT, hot=512, tail=64, pages=64),
        # one layer of decoding at concurrency 8
        _located("attend_decode8", "attend", 8, 1, 2048, 16, LATENT),
        # one layer of speculative verification at concurrency 64
        _located("attend_verify64", "attend", 64, 8, 2048, 16, LATENT),
        # the same layer unsharded, all 128 heads on this GPU, concurrency 16
        _located("attend_heads128", "attend", 16, 8, 2048, 128, LATENT),
        # one request's new token over a 500K-row history: split over length
        _history("attend_500k", "attend", 1, 1, 512000, 16, LATENT),
        # a verify block of 4 on grouped heads in f16, ragged histories
        _history("attend_grouped", "attend", 12, 4, 9000, 32, _grouped(4, 128, 128), ragged=0.9,
                 dtype="f16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _draw_layout(rng):
    if rng.random() < 0.55:
        return dict(LATENT)
    kv = rng.choice([1, 2, 4, 8])
    key = rng.choice([64, 96, 128, 192])
    return _grouped(kv, key, rng.choice([64, 128, key]), rng.choice([0, 0, 16, 32]))


def draw(rng):
    op = rng.choice(["rotate", "append", "store", "read", "attend", "attend", "attend"])
    dtype = rng.choice(["bf16", "bf16", "f16"])
    turn = dict(pairs=rng.choice(["half", "interleaved"]),
                scaling=rng.choice(["plain", "linear", "base", "parts"]), far=_log(rng, 64, 1 << 20))
    if op == "rotate":
        elems = rng.choice([64, 80, 96, 128, 192, 576])
        rotary = rng.choice([16, 32, 64])
        offset = rng.choice([0, elems - rotary])
        heads = _log(rng, 1, 128)
        tokens = _log(rng, 1, max(1, min(16384, (8192 * 32 * 128) // (heads * elems))))
        case = _rotate(None, tokens, heads, elems, offset=offset, rotary=rotary, dtype=dtype, **turn)
    elif op in ("append", "store"):
        layout = _draw_layout(rng)
        wide = layout["wide"]
        # the wide elements turn where there are any that can, else the rest
        rotary = wide or rng.choice([32, 64])
        offset = layout["key"] - wide if wide else 0
        n = layout["kv"] * (layout["key"] + (0 if layout["shared"] else layout["value"]))
        requests = _log(rng, 1, 64) if op == "append" else 1
        tokens = rng.choice([1, 1, 2, 4, 8]) if op == "append" else \
            _log(rng, 16, max(16, min(32768, (16384 * 2048) // n)))
        case = _write(None, op, requests, tokens, layout, rotary=rotary, offset=offset,
                      window=rng.randint(8, 600), dtype=dtype, **turn)
    else:
        layout = _draw_layout(rng)
        kv, latent = layout["kv"], layout["shared"]
        heads = _log(rng, 1, 128) if latent else kv * rng.randint(1, 8)
        n = kv * (layout["key"] + (0 if latent else layout["value"]))
        budget = (110_000_000 if op == "read" else 300_000_000) // n  # rows, as in the listed ones
        if rng.random() < 0.5:
            queries = rng.choice([1, 1, 2, 4, 8])
            topk = _log(rng, 64, 2048)
            requests = max(1, min(64, budget // (queries * topk), _log(rng, 1, 1024) // queries,
                                  (16 * 128) // heads))
            case = _located(None, op, requests, queries, topk, heads, layout,
                            hot=rng.randint(512, 4096), tail=rng.randint(32, 256),
                            pages=rng.randint(64, 512), lost=rng.choice([0.0, 0.0, 0.05]),
                            overlap=rng.choice([0.0, 0.5, 0.8]), dtype=dtype)
        else:
            queries = rng.choice([1, 1, 4, 8]) if op == "attend" else 1
            rows = min(_log(rng, 64, 200000), budget, 30_000_000 // (heads * queries))
            requests = max(1, min(_log(rng, 1, 128), budget // rows,
                                  30_000_000 // (rows * heads * queries)))
            case = _history(None, op, requests, queries, rows, heads, layout,
                            tail=rng.randint(64, 400), ragged=rng.choice([0.0, 0.5, 0.95]),
                            dtype=dtype)
    del case["name"]
    return case


# ------------------------------------------------------------------ layout

def _sizes(c):
    """Where a packed row's parts begin: key codes, value codes, wide elements,
    scales, padding, end."""
    kv, key8 = c["kv"], c["key"] - c["wide"]
    values = 0 if c["shared"] else c["value"]
    at = [0, kv * key8, kv * (key8 + values)]
    at.append(at[2] + 2 * kv * c["wide"])
    at.append(at[3] + 4 * kv * (1 if c["shared"] else 2))
    at.append(-(-at[4] // 16) * 16)
    return at


def _exponent(top):
    """The smallest e with top <= 448 * 2^e, from -64 to 120."""
    m, x = torch.frexp(top)
    e = torch.where(m <= 0.875, x - 9, x - 8)
    return torch.where(top == 0, -64, e).clamp(-64, 120)


def _quantised(x):
    """Codes (as e4m3) and scales of heads [..., n]."""
    e = _exponent(x.abs().amax(-1))
    scale = torch.exp2(e.to(x.dtype))
    return (x / scale[..., None]).to(torch.float8_e4m3fn), scale


def _packed(c, key, wide, value):
    """Rows in bytes: key [..., kv, key8], wide [..., kv, wide] or None, value
    [..., kv, value] or None, in 32 bits."""
    lead = key.shape[:-2]
    code, scale = _quantised(key)
    parts, scales = [code.reshape(*lead, -1).view(torch.uint8)], [scale.float()]
    if value is not None:
        code, scale = _quantised(value)
        parts.append(code.reshape(*lead, -1).view(torch.uint8))
        scales.append(scale.float())
    if wide is not None:
        parts.append(wide.to(TYPES[c["dtype"]]).reshape(*lead, -1).view(torch.uint8))
    parts.append(torch.cat(scales, -1).contiguous().view(torch.uint8))
    at = _sizes(c)
    parts.append(torch.zeros(*lead, at[5] - at[4], dtype=torch.uint8, device=key.device))
    return torch.cat(parts, -1)


def _unpacked(c, rows):
    """Keys [..., kv, key] and values [..., kv, value] of rows in bytes, in 32 bits."""
    kv, at = c["kv"], _sizes(c)
    part = lambda a, b, t: rows[..., a:b].contiguous().view(t).float()  # noqa: E731
    scale = part(at[3], at[4], torch.float32).unflatten(-1, (-1, kv))
    key = part(at[0], at[1], torch.float8_e4m3fn).unflatten(-1, (kv, -1)) * scale[..., 0, :, None]
    value = key[..., :c["value"]] if c["shared"] else \
        part(at[1], at[2], torch.float8_e4m3fn).unflatten(-1, (kv, -1)) * scale[..., 1, :, None]
    if c["wide"]:
        key = torch.cat([key, part(at[2], at[3], TYPES[c["dtype"]]).unflatten(-1, (kv, -1))], -1)
    return key, value


def _frequencies(c):
    """Radians a position of each pair, and what rotated elements are multiplied by."""
    n, base, factor, original, fast, slow = c["rotary"], 10000.0, 8.0, 8192.0, 32.0, 1.0
    if c["scaling"] == "base":
        base *= factor ** (n / (n - 2))
    f = [base ** (-2.0 * i / n) for i in range(n // 2)]
    if c["scaling"] == "linear":
        f = [x / factor for x in f]
    if c["scaling"] == "parts":  # pairs that turn often over the trained length stay as they are
        keep = [min(1.0, max(0.0, (original * x / (2 * math.pi) - slow) / (fast - slow))) for x in f]
        f = [x * k + x / factor * (1 - k) for x, k in zip(f, keep)]
    return f, 0.1 * math.log(factor) + 1 if c["scaling"] == "parts" else 1.0


# ------------------------------------------------------------------ inputs

def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _randn(shape, dtype, g):
    out = torch.empty(shape, dtype=dtype, device=DEV)
    return out.normal_(generator=g)


def _rows(c, n, g):
    """n packed rows of normal elements, each row at a size of its own."""
    at = _sizes(c)
    out = torch.empty((n, at[5]), dtype=torch.uint8, device=DEV)
    kv, step = c["kv"], 1 << 17
    for i in range(0, n, step):
        m = min(step, n - i)
        size = torch.exp2(_randn((m, 1, 1), torch.float32, g) * 0.5)
        x = _randn((m, kv, c["key"]), torch.float32, g) * size
        y = None if c["shared"] else _randn((m, kv, c["value"]), torch.float32, g) * size
        key8 = c["key"] - c["wide"]
        out[i:i + m] = _packed(c, x[..., :key8], x[..., key8:] if c["wide"] else None, y)
    return out


def _positions(c, n, g):
    return torch.randint(0, c["far"], (n,), generator=g, device=DEV, dtype=torch.int32)


def _prep_rotate(c, seed):
    g = _gen(seed)
    x = _randn((c["tokens"], c["heads"], c["elems"]), TYPES[c["dtype"]], g)
    return dict(case=c, x=x, y=torch.empty_like(x), at=_positions(c, c["tokens"], g))


def _prep_write(c, seed):
    g, dt, n = _gen(seed), TYPES[c["dtype"]], c["requests"] * c["tokens"]
    kv, key8 = c["kv"], c["key"] - c["wide"]
    s = dict(case=c, key=_randn((n, kv, key8), dt, g), at=_positions(c, n, g))
    s["wide"] = _randn((n, kv, c["wide"]), dt, g) if c["wide"] else None
    s["value"] = None if c["shared"] else _randn((n, kv, c["value"]), dt, g)
    return s


def _lengths(c, seed):
    """Length of each request's history: `rows`, or down to (1 - ragged) of it."""
    r = random.Random(seed)
    lo = max(1, int(c["rows"] * (1 - c["ragged"])))
    return [c["rows"] if not c["ragged"] else r.randint(lo, c["rows"]) for _ in range(c["requests"])]


def _prep_located(c, seed):
    g = _gen(seed)
    R, Q, k = c["requests"], c["queries"], c["topk"]
    # the tiers (tail, pages, hot) side by side, each 256-byte aligned
    rows = [R * c["tail"], R * c["pages"] * PAGE, R * c["hot"]]
    first, n = [], 0
    for m in rows:
        first.append(n)
        n += -(-m // 16) * 16
    arena = _rows(c, n, g)
    # every request's rows: its tail ring, its pages (scattered slots), its hot slots
    slots = torch.randperm(R * c["pages"], generator=g, device=DEV).view(R, -1, 1)
    r = torch.arange(R, device=DEV).view(R, 1)
    at = lambda m: r * m + torch.arange(m, device=DEV)  # noqa: E731
    pages = (slots * PAGE + torch.arange(PAGE, device=DEV)).view(R, -1)
    every = torch.cat([at(c["tail"]), pages + (1 << 30), at(c["hot"]) + (2 << 30)], 1)
    core = int(c["overlap"] * k) if Q > 1 else 0
    order = torch.rand((R, every.shape[1]), generator=g, device=DEV).argsort(1)
    spare = order[:, core:]
    own_ = torch.arange(Q * (k - core), device=DEV) % spare.shape[1]
    pick = torch.cat([order[:, None, :core].expand(R, Q, core),
                      spare[:, own_].reshape(R, Q, k - core)], 2)
    loc = every.gather(1, pick.reshape(R, -1)).view(R, Q, k)
    loc[torch.rand(loc.shape, generator=g, device=DEV) < c["lost"]] = NO_LOC
    return dict(case=c, arena=arena, tiers=list(zip(first, rows)), g=g,
                first=torch.tensor(first + [0], device=DEV),
                loc=loc.to(torch.int32).contiguous())


def _prep_history(c, seed):
    g, lens = _gen(seed), _lengths(c, seed)
    rows = _rows(c, c["requests"] * c["rows"], g).view(c["requests"], c["rows"], -1)
    return dict(case=c, lens=lens, npages=[n // PAGE for n in lens], history=rows, g=g)


def _prep_over(c, seed):
    s = (_prep_located if c["over"] == "located" else _prep_history)(c, seed)
    dt, g, R, Q = TYPES[c["dtype"]], s.pop("g"), c["requests"], c["queries"]
    if c["op"] == "attend":
        s["q"] = _randn((R, Q, c["heads"], c["key"]), dt, g)
        s["out"] = torch.empty((R, Q, c["heads"], c["value"]), dtype=dt, device=DEV)
        s["lse"] = torch.empty((R, Q, c["heads"]), device=DEV)
    return s


def _inputs(c, seed):
    prep = {"rotate": _prep_rotate, "append": _prep_write, "store": _prep_write}
    return prep.get(c["op"], _prep_over)(c, seed)


def prepare(case, seed):
    s = _inputs(case, seed)
    # what a program keeps between calls: the pool with its arenas, descriptors
    # and workspace, or the same layout in plain tensors
    if own:
        {"rotate": _own_rotate, "append": _own_append, "store": _own_store}.get(case["op"], _own_over)(s)
    else:
        _plain_keep(s)
    torch.cuda.synchronize()
    s.pop("history", None)
    return s


# ------------------------------------------------------- the framework's own

def _layout(c):
    from hierarchical_sparse_kv_dhs_gb300 import dhs
    return dhs.packed_rows(dtype=c["dtype"], kv_heads=c["kv"], key_elems=c["key"],
                           wide_elems=c["wide"], value_elems=c["value"], shared=c["shared"])


def _pool(c, **kw):
    from hierarchical_sparse_kv_dhs_gb300 import dhs
    args = dict(max_requests=1, sources=1, row_bytes=16, page_rows=PAGE, tail_rows=1, hot_rows=16,
                max_queries=1, max_topk=16, max_rows_per_request=64, optional_pages=0)
    if c["op"] != "rotate":
        args["row_bytes"] = dhs.dhs_packed_bytes(_layout(c))
    return dhs.Pool(**{**args, **kw})


def _turns(c):
    """The table of the rotation, on the GPU, and the amplitude."""
    from hierarchical_sparse_kv_dhs_gb300 import dhs
    table = dhs.rope_table(c["rotary"], base=10000.0, scaling=c["scaling"], factor=8.0,
                           original=8192.0, fast=32.0, slow=1.0)
    return torch.from_numpy(table).to(DEV), _frequencies(c)[1]


def _own_rotate(s):
    from hierarchical_sparse_kv_dhs_gb300 import dhs
    c = s["case"]
    s["pool"] = _pool(c)
    s["turns"], a = _turns(c)
    s["st"] = dhs.make_rotate(s["x"], s["at"], s["turns"], out=s["y"], offset=c["offset"],
                              rotary=c["rotary"], pairs=c["pairs"], amplitude=a)


def _own_pack(s, items):
    from hierarchical_sparse_kv_dhs_gb300 import dhs
    c = s["case"]
    s["turns"], a = _turns(c)
    s["st"], s["keep"] = dhs.make_pack(items, _layout(c), rotary_offset=c["offset"],
                                       rotary_elems=c["rotary"], pairs=c["pairs"], amplitude=a,
                                       turns=s["turns"])


def _own_read(s, items):
    from hierarchical_sparse_kv_dhs_gb300 import dhs
    s["rd"], s["keep_rd"] = dhs.make_unpack(items, _layout(s["case"]))


def _read_into(s, *shape):
    c, dt = s["case"], TYPES[s["case"]["dtype"]]
    s["k"] = torch.zeros((*shape, c["kv"], c["key"]), dtype=dt, device=DEV)
    s["v"] = None if c["shared"] else torch.zeros((*shape, c["kv"], c["value"]), dtype=dt, device=DEV)


def _own_store(s):
    from hierarchical_sparse_kv_dhs_gb300 import dhs
    c, n = s["case"], s["case"]["tokens"]
    s["pool"] = _pool(c)
    s["rows"] = torch.empty((n, s["pool"].cfg.row_bytes), dtype=torch.uint8, device=DEV)
    _read_into(s, n)
    _own_pack(s, [dhs.pack_item(n, s["key"], wide=s["wide"], value=s["value"], positions=s["at"],
                                rows=s["rows"])])
    _own_read(s, [dhs.unpack_item(n, s["k"], value=s["v"], rows=s["rows"])])


def _own_append(s):
    from hierarchical_sparse_kv_dhs_gb300 import dhs
    c, R, n = s["case"], s["case"]["requests"], s["case"]["tokens"]
    s["pool"] = _pool(c, max_requests=R, tail_rows=c["window"], page_rows=4096,
                      max_rows_per_request=1 << 19)
    _read_into(s, R, n)
    part = lambda x, r: None if x is None else x[r * n:(r + 1) * n]  # noqa: E731
    items = []
    for r in range(R):
        dhs.check(s["pool"].admit_window(r, 0, None, 0))
        items.append(dhs.pack_item(n, part(s["key"], r), wide=part(s["wide"], r),
                                   value=part(s["value"], r), positions=part(s["at"], r), req=r))
    _own_pack(s, items)
    s["len"] = 0


def _own_over(s):
    from hierarchical_sparse_kv_dhs_gb300 import dhs
    c, R, Q = s["case"], s["case"]["requests"], s["case"]["queries"]
    attend = c["op"] == "attend"
    if c["over"] == "located":
        k, rb = c["topk"], s["arena"].shape[1]
        flat = s["arena"].view(-1)
        tail, opt, hot = [flat[f * rb:(f + m) * rb] for f, m in s["tiers"]]
        s["pool"] = _pool(c, max_requests=R, tail_rows=c["tail"], hot_rows=c["hot"], max_queries=Q,
                          max_topk=k, max_rows_per_request=(c["pages"] + 8) * PAGE,
                          optional_pages=R * c["pages"], arenas=(hot, tail, opt))
        if attend:
            items = [dhs.attend_item(queries=Q, topk=k, q=s["q"][r], loc=s["loc"][r],
                                     out=s["out"][r], lse=s["lse"][r]) for r in range(R)]
        else:
            _read_into(s, R, Q, k)
            items = [dhs.unpack_item(Q * k, s["k"][r], value=None if c["shared"] else s["v"][r],
                                     loc=s["loc"][r]) for r in range(R)]
    else:
        lens, rb = s["lens"], s["history"].shape[2]
        s["pool"] = _pool(c, max_requests=R, tail_rows=c["tail"], max_queries=Q,
                          max_rows_per_request=c["rows"], optional_pages=sum(s["npages"]))
        s["host"] = torch.empty((R, c["rows"] * rb), dtype=torch.uint8, pin_memory=True)
        for r, n in enumerate(lens):
            dhs.check(s["pool"].admit_device(r, 0, s["history"][r].data_ptr(),
                                             s["host"][r].data_ptr(), n)[0])
        dhs.check(s["pool"].flush())
        if attend:
            items = [dhs.attend_item(req=r, queries=Q, flags=dhs.DHS_ATTEND_HISTORY, q=s["q"][r],
                                     out=s["out"][r], lse=s["lse"][r]) for r in range(R)]
        else:
            _read_into(s, R, c["rows"])
            items = [dhs.unpack_item(n, s["k"][r], value=None if c["shared"] else s["v"][r], req=r,
                                     first=0, flags=dhs.DHS_UNPACK_HISTORY) for r, n in enumerate(lens)]
    if not attend:
        return _own_read(s, items)
    s["st"], s["keep"] = dhs.make_attend_packed(items, _layout(c), heads=c["heads"],
                                                scale=c["key"] ** -0.5)
    s["work"] = torch.zeros(max(256, s["pool"].attend_packed_bytes(s["st"])), dtype=torch.uint8, device=DEV)
    s["st"].work_dev, s["st"].work_bytes = s["work"].data_ptr(), s["work"].numel()


def _run_own(s):
    from hierarchical_sparse_kv_dhs_gb300 import dhs
    c, pool = s["case"], s["pool"]
    if c["op"] == "rotate":
        dhs.check(pool.rotate(s["st"]), "dhs_rotate")
        return [s["y"]]
    if c["op"] == "attend":
        dhs.check(pool.attend_packed(s["st"]), "dhs_attend_packed")
        return [s["out"], s["lse"]]
    if c["op"] == "store":
        dhs.check(pool.pack(s["st"]), "dhs_pack")
    if c["op"] == "append":
        n = c["tokens"]
        if s["len"] + n > 1 << 19:  # as long as a request may get: the next one
            for r in range(c["requests"]):
                dhs.check(pool.release(r), "dhs_release")
                dhs.check(pool.admit_window(r, 0, None, 0), "dhs_admit_window")
            s["len"] = 0
        dhs.check(pool.append_packed(s["st"]), "dhs_append_packed")
        _own_read(s, [dhs.unpack_item(n, s["k"][r], value=None if c["shared"] else s["v"][r], req=r,
                                      first=s["len"], flags=dhs.DHS_UNPACK_HISTORY)
                      for r in range(c["requests"])])
        s["len"] += n
    dhs.check(pool.unpack(s["rd"]), "dhs_unpack")
    return [s["k"]] if c["shared"] else [s["k"], s["v"]]


# ------------------------------------------------------------- plain forms

def _plain_keep(s):
    """What the plain forms keep: the rotation's frequencies, a window's ring,
    a history's pages in one arena with the tail rings behind them."""
    c = s["case"]
    if c["op"] in ("rotate", "append", "store"):
        f, s["amplitude"] = _frequencies(c)
        s["freq"] = torch.tensor(f, dtype=torch.float64, device=DEV)
    if c["op"] == "append":
        s["ring"] = torch.zeros((c["requests"], c["window"], _sizes(c)[5]), dtype=torch.uint8, device=DEV)
        s["len"] = 0
    if c.get("over") != "history":
        return
    R, T, lens = c["requests"], c["tail"], s["lens"]
    total, first = sum(s["npages"]), 0
    s["arena"] = torch.zeros((total * PAGE + R * T, s["history"].shape[2]), dtype=torch.uint8, device=DEV)
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


def _turned(c, s, x):
    """x [n, heads, rotary] in 32 bits, its pairs turned by position * frequency
    (angles in 64 bits: far positions) and multiplied by the amplitude."""
    angle = s["at"].double()[:, None] * s["freq"]
    co = (torch.cos(angle) * s["amplitude"]).float()[:, None]
    si = (torch.sin(angle) * s["amplitude"]).float()[:, None]
    if c["pairs"] == "half":
        a, b = x.chunk(2, -1)
        return torch.cat([a * co - b * si, b * co + a * si], -1)
    a, b = x[..., 0::2], x[..., 1::2]
    return torch.stack([a * co - b * si, b * co + a * si], -1).flatten(-2)


def _plain_rotate(s):
    c, x = s["case"], s["x"]
    o, n = c["offset"], c["rotary"]
    return [torch.cat([x[..., :o], _turned(c, s, x[..., o:o + n].float()).to(x.dtype), x[..., o + n:]], -1)]


def _plain_pack(s):
    c, o, n = s["case"], s["case"]["offset"], s["case"]["rotary"]
    key8 = c["key"] - c["wide"]
    key, wide = s["key"].float(), None if s["wide"] is None else s["wide"].float()
    if o >= key8:
        o -= key8
        wide = torch.cat([wide[..., :o], _turned(c, s, wide[..., o:o + n]), wide[..., o + n:]], -1)
    else:
        key = torch.cat([key[..., :o], _turned(c, s, key[..., o:o + n]), key[..., o + n:]], -1)
    return _packed(c, key, wide, None if s["value"] is None else s["value"].float())


def _read_out(c, rows, keep=None):
    key, value = _unpacked(c, rows)
    dt = TYPES[c["dtype"]]
    if keep is not None:
        key, value = key.masked_fill(~keep[..., None, None], 0), value.masked_fill(~keep[..., None, None], 0)
    return [key.to(dt)] if c["shared"] else [key.to(dt), value.to(dt)]


def _plain_append(s):
    c, R, n, T = s["case"], s["case"]["requests"], s["case"]["tokens"], s["case"]["window"]
    slot = (s["len"] + torch.arange(n, device=DEV)) % T
    s["ring"][:, slot] = _plain_pack(s).view(R, n, -1)
    s["len"] += n
    return _read_out(c, s["ring"][:, slot])


def _attention(q, k, v, keep, scale):
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


def _by_heads(c, q, rows, keep):
    """Attention of q [b, Q, H, d] over packed rows [b, n, bytes] by groups of heads; keep [b, Q, n]."""
    b, Q, H = q.shape[:3]
    G, n = c["kv"], rows.shape[1]
    k, v = (x.permute(2, 0, 1, 3).reshape(G * b, n, -1) for x in _unpacked(c, rows))
    q = q.view(b, Q, G, H // G, -1).permute(2, 0, 1, 3, 4).reshape(G * b, Q * H // G, -1)
    keep = keep[None, :, :, None].expand(G, b, Q, H // G, n).reshape(G * b, Q * H // G, n)
    o, lse = _attention(q, k, v, keep, c["key"] ** -0.5)
    o = o.view(G, b, Q, H // G, -1).permute(1, 2, 0, 3, 4).reshape(b * Q, H, -1)
    return o, lse.view(G, b, Q, H // G).permute(1, 2, 0, 3).reshape(b * Q, H)


def _joined(outs, s):
    o, lse = (torch.cat(x) for x in zip(*outs))
    return [o.view(s["out"].shape).to(s["out"].dtype), lse.view(s["lse"].shape)]


def _plain_located(s):
    c, attend = s["case"], s["case"]["op"] == "attend"
    R, Q, k = s["loc"].shape
    outs = []
    for r in range(0, R, 16):  # the selected rows of 16 requests at a time
        loc = s["loc"][r:r + 16].long() & 0xFFFFFFFF
        keep = loc < 0xC0000000
        at = torch.where(keep, s["first"][loc >> 30] + (loc & 0x3FFFFFFF), 0)
        b, rows = len(loc), s["arena"][at]
        if attend:
            q = s["q"][r:r + 16].float().view(b * Q, 1, c["heads"], -1)
            outs.append(_by_heads(c, q, rows.view(b * Q, k, -1), keep.view(b * Q, 1, -1)))
        else:
            outs.append(_read_out(c, rows, keep))
    return _joined(outs, s) if attend else [torch.cat(x) for x in zip(*outs)]


def _plain_history(s):
    c, attend = s["case"], s["case"]["op"] == "attend"
    R, Q, T = c["requests"], c["queries"], c["tail"]
    pos = torch.arange(0, max(s["lens"]) if attend else c["rows"], device=DEV)
    outs = []
    elems = c["kv"] * (c["key"] + c["value"])
    per = max(1, 600_000_000 // (len(pos) * elems))
    for r in range(0, R, per):  # as many histories at a time as fit in 2.4 GB
        n, tab = s["len"][r:r + per, None], s["table"][r:r + per]
        page = tab[:, (pos // PAGE).clamp(max=tab.shape[1] - 1)] * PAGE + pos % PAGE
        at = torch.where(pos >= n - T, s["ring"][r:r + per, None] + pos % T, page)
        rows = s["arena"][at]
        if attend:
            # query i of the block is the row L - Q + i: it sees itself and what precedes it
            end = n - (Q - 1) + torch.arange(Q, device=DEV)
            outs.append(_by_heads(c, s["q"][r:r + per].float(), rows, pos < end[..., None]))
        else:
            outs.append(_read_out(c, rows, pos < n))
    return _joined(outs, s) if attend else [torch.cat(x) for x in zip(*outs)]


def run(state):
    if own:
        return _run_own(state)
    c = state["case"]
    if c["op"] == "rotate":
        return _plain_rotate(state)
    if c["op"] == "append":
        return _plain_append(state)
    if c["op"] == "store":
        return _read_out(c, _plain_pack(state))
    return (_plain_located if c["over"] == "located" else _plain_history)(state)


# ------------------------------------------------------------ work and truth

def work(case):
    c = case
    if c["op"] == "rotate":
        return {"bytes": c["tokens"] * (4 * c["heads"] * c["elems"] + 4) + 4 * c["rotary"],
                "flops": 3 * c["tokens"] * c["heads"] * c["rotary"]}
    packed = _sizes(c)[5]
    wide = 2 * c["kv"] * (c["key"] + (0 if c["shared"] else c["value"]))  # a row in 16 bits
    if c["op"] in ("append", "store"):
        n = c["requests"] * c["tokens"]
        return {"bytes": n * (2 * wide + 2 * packed + 4) + 4 * c["rotary"],
                "flops": n * (wide + 3 * c["kv"] * c["rotary"])}
    R, Q = c["requests"], c["queries"]
    if c["over"] == "located":
        k = c["topk"]
        core = int(c["overlap"] * k) if Q > 1 else 0
        spare = R * (c["tail"] + c["pages"] * PAGE + c["hot"] - core)
        rows = (R * core + min(spare, R * Q * (k - core))) * (1 - c["lost"])
        read, pairs, io = R * Q * k, Q * R * k * (1 - c["lost"]), 4 * R * Q * k
    else:
        rows = R * c["rows"] * (1 - c["ragged"] / 2)
        read, pairs, io = R * c["rows"], rows * Q, 0
    if c["op"] == "read":
        return {"bytes": rows * packed + io + read * wide, "flops": pairs * wide / 2}
    heads = R * Q * c["heads"]
    io += heads * (2 * (c["key"] + c["value"]) + 4)
    return {"bytes": rows * packed + io, "flops": 2 * pairs * c["heads"] * (c["key"] + c["value"])}


def _number(codes):
    """What e4m3 codes (bytes) stand for, in 64 bits."""
    b = codes.long()
    e, m = (b >> 3) & 15, (b & 7).double()
    x = torch.where(e == 0, m * 2.0 ** -9, (8 + m) * torch.exp2((e - 10).double()))
    x = torch.where((b & 127) == 127, float("nan"), x)
    return torch.where(b >= 128, -x, x)


def _true_rows(c, rows):
    """Keys and values of packed rows [n, bytes] in 64 bits, head by head."""
    at, kv, key8 = _sizes(c), c["kv"], c["key"] - c["wide"]
    scale = rows[:, at[3]:at[4]].contiguous().view(torch.float32).double()
    keys, values = [], []
    for g in range(kv):
        x = _number(rows[:, g * key8:(g + 1) * key8]) * scale[:, g:g + 1]
        if c["shared"]:
            values.append(x[:, :c["value"]])
        else:
            lo = at[1] + g * c["value"]
            values.append(_number(rows[:, lo:lo + c["value"]]) * scale[:, kv + g:kv + g + 1])
        if c["wide"]:
            lo = at[2] + 2 * g * c["wide"]
            w = rows[:, lo:lo + 2 * c["wide"]].contiguous().view(TYPES[c["dtype"]]).double()
            x = torch.cat([x, w], 1)
        keys.append(x)
    return keys, values


def _true_turn(c, at, x):
    """x [n, heads, rotary] as complex numbers turned by e^(i angle)."""
    f, a = _frequencies(c)
    angle = at.double()[:, None, None] * torch.tensor(f, dtype=torch.float64, device=DEV)
    x = x.double()
    z = torch.complex(x[..., :len(f)].contiguous(), x[..., len(f):].contiguous()) if c["pairs"] == "half" \
        else torch.view_as_complex(x.unflatten(-1, (-1, 2)).contiguous())
    z = z * torch.polar(torch.full_like(angle, a), angle)
    return torch.cat([z.real, z.imag], -1) if c["pairs"] == "half" else torch.view_as_real(z).flatten(-2)


def _true_rounded(x):
    """x [..., n] in 64 bits as a head of codes holds it: to 4 bits of
    significand, ties to even, in steps of at least 2^-9 of the scale."""
    top = x.abs().amax(-1, keepdim=True)
    e = torch.ceil(torch.log2(top.clamp(min=1e-300) / 448))
    e = torch.where(top > 448 * torch.exp2(e), e + 1, torch.where(top <= 448 * torch.exp2(e - 1), e - 1, e))
    scale = torch.exp2(e.clamp(-64, 120))
    y = x / scale
    size = torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6)))
    size = torch.where(torch.exp2(size) > y.abs().clamp(min=2.0 ** -6), size - 1, size)
    step = torch.exp2(size - 3)
    return torch.round(y / step) * step * scale


def _exact_rotate(c, s):
    y = s["x"].double()
    o, n = c["offset"], c["rotary"]
    y[..., o:o + n] = _true_turn(c, s["at"], s["x"][..., o:o + n])
    return [y]


def _exact_write(c, s):
    o, n, key8 = c["offset"], c["rotary"], c["key"] - c["wide"]
    key = torch.cat([s["key"], s["wide"]], -1).double() if c["wide"] else s["key"].double()
    key[..., o:o + n] = _true_turn(c, s["at"], key[..., o:o + n])
    key[..., :key8] = _true_rounded(key[..., :key8])
    lead = (c["requests"], c["tokens"]) if c["op"] == "append" else (c["tokens"],)
    outs = [key] if c["shared"] else [key, _true_rounded(s["value"].double())]
    return [x.view(*lead, *x.shape[1:]) for x in outs]


def exact(case, seed):
    c = case
    s = _inputs(c, seed)
    if c["op"] == "rotate":
        return _exact_rotate(c, s)
    if c["op"] in ("append", "store"):
        return _exact_write(c, s)
    attend, R, Q = c["op"] == "attend", c["requests"], c["queries"]
    shape = (R, Q, c["topk"]) if c["over"] == "located" else (R, c["rows"])
    if attend:
        out = torch.zeros(s["out"].shape, dtype=torch.float64, device=DEV)
        lse = torch.full(s["lse"].shape, float("-inf"), dtype=torch.float64, device=DEV)
    else:
        k = torch.zeros((*shape, c["kv"], c["key"]), dtype=torch.float64, device=DEV)
        v = None if c["shared"] else torch.zeros((*shape, c["kv"], c["value"]), dtype=torch.float64, device=DEV)
    share = c["heads"] // c["kv"]
    for r in range(R):
        for i in range(Q):
            if c["over"] == "located":
                loc = s["loc"][r, i].long() & 0xFFFFFFFF
                there = (loc != NO_LOC).nonzero()[:, 0]
                loc = loc[there]
                rows = s["arena"][s["first"][loc >> 30] + (loc & 0x3FFFFFFF)]
            else:
                n = s["lens"][r] - (Q - 1 - i if attend else 0)
                there = torch.arange(max(0, n), device=DEV)
                rows = s["history"][r, :max(0, n)]
            if not len(rows):
                continue
            keys, values = _true_rows(c, rows)
            for g in range(c["kv"]):
                if attend:
                    h = slice(g * share, (g + 1) * share)
                    x = s["q"][r, i, h].double() @ keys[g].T / math.sqrt(c["key"])
                    lse[r, i, h] = torch.logsumexp(x, 1)
                    out[r, i, h] = torch.softmax(x, 1) @ values[g]
                else:
                    at = (r, i) if c["over"] == "located" else (r,)
                    k[at][there, g] = keys[g]
                    if v is not None:
                        v[at][there, g] = values[g]
    if attend:
        return [out, lse]
    return [k] if v is None else [k, v]
