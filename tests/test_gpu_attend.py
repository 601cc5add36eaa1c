"""dhs_attend against the formula in 64 bits: located rows (all three tiers,
entries without a row, union lists) and histories (ring, pages, host rows,
windows), over head layouts, lengths and masks where a tiled, split kernel can
go wrong.

Bounds, from the number formats alone.  With unit roundoff u of the row type
(bf16 2^-8, f16 2^-11), weights w_j summing to 1 and A = sum w_j |y_j|: the
rounding of the weights moves the output by at most u A, its own rounding by
u |out|, and a score error d (float accumulation of dk products in steps of
at least 8: d <= 2^-22 (dk / 8 + 8) max_j scale sum |q x_j|) by 2 d A.  An f16
weight below the subnormal step is lost whole: n 2^-25 max |y|.  The log-sum
is off by at most d, plus the roundings of its own logarithm and sum.
"""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

U = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11}
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16}
PAGE = 16
NAN = float("nan")


@pytest.fixture(scope="module")
def dhs():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from hierarchical_sparse_kv_dhs_gb300.build import build
    build()
    from hierarchical_sparse_kv_dhs_gb300 import dhs as mod
    return mod


class Layout:
    def __init__(self, heads, key, value, kv=1, key_offset=0, value_offset=0, elems=None,
                 key_stride=None, value_stride=None, dtype="bf16"):
        self.heads, self.key, self.value, self.kv, self.dtype = heads, key, value, kv, dtype
        self.key_offset, self.value_offset = key_offset, value_offset
        self.key_stride = key if key_stride is None else key_stride
        self.value_stride = value if value_stride is None else value_stride
        self.elems = elems or max(key_offset + (kv - 1) * self.key_stride + key,
                                  value_offset + (kv - 1) * self.value_stride + value)
        self.scale = key ** -0.5

    def args(self):
        return dict(heads=self.heads, kv_heads=self.kv, key_elems=self.key, value_elems=self.value,
                    key_offset=self.key_offset, value_offset=self.value_offset,
                    key_stride=self.key_stride, value_stride=self.value_stride,
                    scale=self.scale, dtype=self.dtype)


LAYOUTS = {
    "latent": Layout(16, 576, 512),
    "latent_f16": Layout(24, 576, 512, dtype="f16"),
    "latent_one_head": Layout(1, 576, 512),
    "latent_64": Layout(64, 576, 512),
    "latent_128": Layout(128, 576, 512),
    "latent_100": Layout(100, 576, 512),
    "grouped": Layout(40, 128, 128, kv=8, value_offset=1024),
    "grouped_f16": Layout(6, 96, 64, kv=2, value_offset=192, dtype="f16"),
    "interleaved": Layout(8, 64, 128, kv=4, value_offset=64, key_stride=192, value_stride=192),
    "smallest": Layout(3, 8, 8),
    "odd": Layout(17, 72, 40, value_offset=24, elems=88),
    "same": Layout(33, 64, 64),
    "largest": Layout(20, 576, 512, value_offset=576, elems=1088),
    "value_only_shift": Layout(5, 200, 200, key_offset=8, value_offset=16),
}




def reference(lay, q, rows, keep):
    """Outputs and bounds in 64 bits: q [Q, H, dk], rows [Q or 1, n, E], keep [Q, n]."""
    Q, H = q.shape[:2]
    share, u = H // lay.kv, U[lay.dtype]
    out = torch.zeros(Q, H, lay.value, dtype=torch.float64, device=q.device)
    lse = torch.full((Q, H), -math.inf, dtype=torch.float64, device=q.device)
    tol, ltol = torch.zeros_like(out), torch.zeros_like(lse)
    for i in range(Q):
        r = rows[i if rows.shape[0] > 1 else 0][keep[i]].double()
        if len(r) == 0:
            continue
        for g in range(lay.kv):
            hs = slice(g * share, (g + 1) * share)
            ko, vo = lay.key_offset + g * lay.key_stride, lay.value_offset + g * lay.value_stride
            x, y, qg = r[:, ko:ko + lay.key], r[:, vo:vo + lay.value], q[i, hs].double()
            s = qg @ x.T * lay.scale
            m = s.amax(1, keepdim=True)
            p = torch.exp(s - m.masked_fill(m == -math.inf, 0))
            z = p.sum(1, keepdim=True)
            w = p / z.masked_fill(z == 0, 1)
            out[i, hs], lse[i, hs] = w @ y, (m + torch.log(z))[:, 0]
            big = (qg.abs() @ x.abs().T).masked_fill(w == 0, 0).amax(1, keepdim=True) * lay.scale
            d = 2.0 ** -22 * (lay.key / 8 + 8) * big
            tol[i, hs] = (1.02 * u + 2 * d) * (w @ y.abs()) + 1.02 * u * out[i, hs].abs() + 2.0 ** -25
            if lay.dtype == "f16":
                tol[i, hs] += len(r) * 2.0 ** -25 * y.abs().max()
            ltol[i, hs] = d[:, 0] + 2.0 ** -21 * (lse[i, hs].abs() + 1)
    return out, lse, tol, ltol


def compare(lay, q, rows, keep, out, lse):
    ro, rl, tol, ltol = reference(lay, q, rows, keep)
    err = (out.double() - ro).abs()
    assert bool((err <= tol).all()), f"output off by {(err / tol.clamp(min=1e-300)).max():.3g} bounds"
    none = rl == -math.inf
    assert torch.equal(none, lse == -math.inf)
    assert bool((out[none] == 0).all())
    e = (lse.double() - rl).abs()
    assert bool((e[~none] <= ltol[~none]).all()), f"log-sum off by {(e / ltol)[~none].max():.3g} bounds"


def run(dhs, pool, lay, items, stream=None, **kw):
    st, keep = dhs.make_attend(items, **{**lay.args(), **kw})
    work = torch.empty(max(256, pool.attend_bytes(st)), dtype=torch.uint8, device="cuda").fill_(0xA5)
    st.work_dev, st.work_bytes = work.data_ptr(), work.numel()
    rc = pool.attend_on(st, stream.cuda_stream) if stream else pool.attend(st)
    assert rc == 0, dhs.lib.dhs_strerror(rc)
    return work


class Located:
    """A pool with caller-given arenas of random rows, and location vectors."""

    def __init__(self, dhs, lay, R=3, T=20, B=50, pages=30, seed=0, sources=1):
        self.dhs, self.lay = dhs, lay
        self.g = torch.Generator("cuda").manual_seed(seed)
        rb = lay.elems * 2
        self.sizes = [R * sources * B, R * sources * T, pages * PAGE]  # hot, tail, opt
        self.arenas = [torch.randn(n, lay.elems, generator=self.g, device="cuda").to(TYPES[lay.dtype])
                       for n in self.sizes]
        flat = [a.view(torch.uint8).view(-1) for a in self.arenas]
        self.pool = dhs.Pool(max_requests=R, sources=sources, row_bytes=rb, page_rows=PAGE,
                             tail_rows=T, hot_rows=B, max_queries=8, max_topk=64,
                             max_rows_per_request=4096, optional_pages=pages, arenas=flat)

    def rand_loc(self, Q, k):
        """Random locations of every tier: (uint32 as int64 [Q, k])."""
        hot, tail, opt = self.sizes
        tier = torch.randint(0, 3, (Q, k), generator=self.g, device="cuda")
        n = torch.tensor([tail, opt, hot], device="cuda")[tier]
        return (tier << 30) + (torch.rand(Q, k, generator=self.g, device="cuda") * n).long()

    def rows(self, loc):
        """The rows [Q, k, E] at `loc` and whether each is one."""
        keep = loc < 0xC0000000
        tier, x = torch.where(keep, loc >> 30, 0), torch.where(keep, loc & 0x3FFFFFFF, 0)
        hot, tail, opt = self.arenas
        every = torch.cat([tail, opt, hot])
        first = torch.tensor([0, len(tail), len(tail) + len(opt)], device="cuda")
        return every[first[tier] + x], keep

    def poison(self, loc):
        """NaN and infinities in every row that no location names."""
        hot, tail, opt = self.arenas
        for t, a in ((0, tail), (1, opt), (2, hot)):
            named = torch.zeros(len(a), dtype=torch.bool, device="cuda")
            named[(loc[(loc < 0xC0000000) & (loc >> 30 == t)] & 0x3FFFFFFF)] = True
            a[~named] = NAN
            a[~named, ::3] = math.inf

    def item(self, loc, index=None, seed=None):
        Q, k = loc.shape
        lay = self.lay
        q = torch.randn(Q, lay.heads, lay.key, generator=self.g, device="cuda").to(TYPES[lay.dtype])
        out = torch.full((Q, lay.heads, lay.value), 7.0, dtype=q.dtype, device="cuda")
        lse = torch.full((Q, lay.heads), 7.0, device="cuda")
        keep = loc.to(torch.int32).contiguous()
        it = self.dhs.attend_item(queries=Q, topk=k, q=q, loc=keep, index=index, out=out, lse=lse)
        return it, (q, out, lse, keep)


def check_located(env, cases):
    """cases: (loc [Q, k] as int64, tensors of item())."""
    torch.cuda.synchronize()
    for loc, (q, out, lse, _) in cases:
        rows, keep = env.rows(loc)
        compare(env.lay, q, rows, keep, out, lse)


@pytest.mark.parametrize("k", [0, 1, 2, 31, 127, 128, 129, 300])
@pytest.mark.parametrize("name", sorted(LAYOUTS))
def test_located_layouts_and_lengths(dhs, name, k):
    env = Located(dhs, LAYOUTS[name], seed=k)
    cases, items = [], []
    for Q in (1, 3):
        loc = env.rand_loc(Q, k)
        it, t = env.item(loc)
        items.append(it)
        cases.append((loc, t))
    env.poison(torch.cat([c[0].reshape(-1) for c in cases]))
    run(dhs, env.pool, env.lay, items)
    check_located(env, cases)
    assert env.pool.status() == (0, 0)


@pytest.mark.parametrize("name", ["latent", "latent_64", "grouped_f16", "odd"])
@pytest.mark.parametrize("k", [1, 40, 260])
def test_located_masks(dhs, name, k):
    """Entries without a row: some, whole queries, whole tiles, first and last ones."""
    env = Located(dhs, LAYOUTS[name], seed=5)
    loc = env.rand_loc(6, k)
    drop = torch.rand(6, k, generator=env.g, device="cuda") < 0.4
    drop[1] = True                    # nothing to attend
    drop[2, : k - 1] = True           # the last entry only
    drop[3, 1:] = True                # the first entry only
    drop[4, : min(k, 128)] = True     # the whole first tile (k = 1, 40: everything)
    loc[drop] = 0xFFFFFFFF
    loc[5, k // 2:] = 0xFFFFFFFE      # past the end of a list
    it, t = env.item(loc)
    env.poison(loc.reshape(-1))
    run(dhs, env.pool, env.lay, [it])
    check_located(env, [(loc, t)])
    assert bool((t[1][1] == 0).all()) and bool((t[2][1] == -math.inf).all())
    assert env.pool.status() == (0, 0)


def test_located_long_selection_split_over_blocks(dhs):
    """One query over 5000 entries (duplicates included) is split and joined;
    the same call twice gives the same bits."""
    for name in ("latent", "latent_128", "grouped"):
        env = Located(dhs, LAYOUTS[name], seed=9)
        loc = env.rand_loc(1, 5000)
        it, t = env.item(loc)
        run(dhs, env.pool, env.lay, [it])
        check_located(env, [(loc, t)])
        first = t[1].clone(), t[2].clone()
        run(dhs, env.pool, env.lay, [it])
        torch.cuda.synchronize()
        assert torch.equal(first[0], t[1]) and torch.equal(first[1], t[2])


@pytest.mark.parametrize("items", [1, 17, 250])
def test_located_ragged_items(dhs, items):
    """Items of different Q and k in one step, more than one launch table."""
    env = Located(dhs, LAYOUTS["odd"], seed=items)
    cases, its = [], []
    for i in range(items):
        loc = env.rand_loc(i % 4, (37 * i) % 290)
        it, t = env.item(loc)
        its.append(it)
        cases.append((loc, t))
    run(dhs, env.pool, env.lay, its)
    check_located(env, [c for c in cases if c[0].shape[0]])


def test_located_union_index(dhs):
    """A union list with per-query positions; negative positions are no row."""
    env = Located(dhs, LAYOUTS["latent"], seed=3)
    Q, k, U_ = 4, 150, 200
    lst = env.rand_loc(1, Q * k).view(Q, k)
    flat = lst.view(-1)
    flat[U_:] = 0xFFFFFFFE
    index = torch.randint(0, U_, (Q, k), generator=env.g, device="cuda")
    index[torch.rand(Q, k, generator=env.g, device="cuda") < 0.2] = -1
    index[2] = -1
    idx32 = index.to(torch.int32)
    it, t = env.item(lst, index=idx32)
    run(dhs, env.pool, env.lay, [it])
    seen = torch.where(index >= 0, flat[index.clamp(min=0)], 0xFFFFFFFF)
    check_located(env, [(seen, t)])
    assert env.pool.status() == (0, 0)
    idx32[0, 0], idx32[1, 1] = Q * k, 2 ** 31 - 1  # past the list
    seen[0, 0] = seen[1, 1] = 0xFFFFFFFF
    run(dhs, env.pool, env.lay, [it])
    check_located(env, [(seen, t)])
    assert env.pool.status() == (dhs.DHS_ERANGE, dhs.DHS_STATUS_ELOC)


def test_located_out_of_arena(dhs):
    """Locations outside their arena take no part and raise ELOC."""
    env = Located(dhs, LAYOUTS["grouped"], seed=4)
    loc = env.rand_loc(2, 140)
    hot, tail, opt = env.sizes
    it, t = env.item(loc)
    for e, bad in ((0, tail), (5, (1 << 30) + opt), (139, (2 << 30) + hot), (7, 0xC0000000)):
        t[3][1, e] = torch.tensor(bad, device="cuda").to(torch.int32)
        loc[1, e] = 0xFFFFFFFF
    run(dhs, env.pool, env.lay, [it])
    check_located(env, [(loc, t)])
    assert env.pool.status() == (dhs.DHS_ERANGE, dhs.DHS_STATUS_ELOC)
    assert env.pool.status() == (0, 0)


def _directed(env, loc, scores, t):
    """Rows named by `loc` [1, k] whose score is about scores[j] for every head."""
    lay = env.lay
    q = t[0]
    q.zero_()
    q[..., 0] = 1.0
    hot, tail, opt = env.arenas
    for t_, a in ((0, tail), (1, opt), (2, hot)):
        at = (loc[0] >> 30) == t_
        x = loc[0][at] & 0x3FFFFFFF
        for g in range(lay.kv):
            a[x, lay.key_offset + g * lay.key_stride] = (scores[at] / lay.scale).to(a.dtype)


@pytest.mark.parametrize("name", ["latent", "latent_64", "grouped", "grouped_f16"])
@pytest.mark.parametrize("shape", ["rising", "falling", "spike", "wide"])
def test_located_score_ranges(dhs, name, shape):
    """Scores whose maximum moves all the time, or by much more than exp's range."""
    env = Located(dhs, LAYOUTS[name], seed=6)
    k = 600
    n = torch.arange(k, device="cuda", dtype=torch.float32)
    scores = {"rising": n / 4 - 70, "falling": 70 - n / 4, "spike": torch.where(n == 401, 300.0, -300.0),
              "wide": (n * 37 % k) - 300}[shape]
    # distinct rows, so that every entry has the score meant for it
    order = torch.randperm(sum(env.sizes), generator=env.g, device="cuda")[:k]
    hot, tail, opt = env.sizes
    loc = torch.where(order < tail, order, torch.where(order < tail + opt, order - tail + (1 << 30),
                                                       order - tail - opt + (2 << 30)))[None]
    it, t = env.item(loc)
    _directed(env, loc, scores, t)
    run(dhs, env.pool, env.lay, [it])
    check_located(env, [(loc, t)])


@pytest.mark.parametrize("low", [-math.inf, "lowest"])
def test_located_scores_at_the_bottom(dhs, low):
    """Scores of -infinity weigh nothing; only such scores: zeros.  Scores of
    the type's lowest value are scores like others."""
    env = Located(dhs, LAYOUTS["grouped_f16"], seed=8)
    hot, tail, opt = env.sizes
    k = 200
    loc = (torch.randperm(opt, generator=env.g, device="cuda")[:k] + (1 << 30))[None].repeat(2, 1)
    it, t = env.item(loc)
    v = -65504.0 if low == "lowest" else low
    scores = torch.where(torch.arange(k, device="cuda") % 3 == 0, 0.5, v)
    lay = env.lay
    q = t[0]
    q.zero_()
    q[..., 0] = 1.0
    x = loc[0] & 0x3FFFFFFF
    for g in range(lay.kv):
        env.arenas[2][x, lay.key_offset + g * lay.key_stride] = scores.half()
        env.arenas[2][x, lay.key_offset + g * lay.key_stride + 1:lay.key_offset + (g + 1) * lay.key_stride] = 0
    if low != "lowest":
        t[3][1, ::3] = -1  # the second query attends scores of -infinity only
        loc[1, ::3] = 0xFFFFFFFF
    else:
        t[3][1, ::3] = -1
        loc[1, ::3] = 0xFFFFFFFF
    run(dhs, env.pool, env.lay, [it])
    check_located(env, [(loc, t)])


def test_located_not_a_number_stays_with_its_query(dhs):
    """A row with NaN makes the queries that attend it NaN, and no other."""
    env = Located(dhs, LAYOUTS["latent"], seed=2)
    loc = env.rand_loc(3, 200)
    bad = env.sizes[2] - 1 + (1 << 30)
    loc[loc == bad] = 0
    loc[1, 77] = bad
    it, t = env.item(loc)
    env.arenas[2][-1] = NAN
    run(dhs, env.pool, env.lay, [it])
    torch.cuda.synchronize()
    assert bool(t[1][1].isnan().all()) and bool(t[2][1].isnan().all())
    rows, keep = env.rows(loc)
    for i in (0, 2):
        compare(env.lay, t[0][i:i + 1], rows[i:i + 1], keep[i:i + 1], t[1][i:i + 1], t[2][i:i + 1])


def test_strides_alignment_and_missing_log_sum(dhs):
    """Queries and outputs as [H][Q] slices of wider, misaligned buffers;
    nothing outside the outputs is written."""
    lay = LAYOUTS["grouped"]
    env = Located(dhs, lay, seed=7)
    Q, k = 3, 70
    loc = env.rand_loc(Q, k)
    lt = loc.to(torch.int32).contiguous()
    for off in (0, 1, 5):
        qb = torch.randn(lay.heads * Q * 150 + 8, generator=env.g, device="cuda").bfloat16()
        ob = torch.full((lay.heads * Q * 140 + 8,), 3.0, device="cuda").bfloat16()
        q = torch.as_strided(qb, (Q, lay.heads, lay.key), (150, Q * 150, 1), off)
        o = torch.as_strided(ob, (Q, lay.heads, lay.value), (140, Q * 140, 1), off)
        it = dhs.attend_item(queries=Q, topk=k, q=qb.data_ptr() + 2 * off, loc=lt,
                             out=ob.data_ptr() + 2 * off)
        run(dhs, env.pool, lay, [it], q_strides=(150, Q * 150), out_strides=(140, Q * 140))
        torch.cuda.synchronize()
        rows, keep = env.rows(loc)
        ro, rl, tol, _ = reference(lay, q, rows, keep)
        assert bool(((o.double() - ro).abs() <= tol).all())
        o.fill_(3.0)
        assert bool((ob == 3.0).all())


def test_shared_query_head_stride_zero(dhs):
    """A head stride of 0: every head asks the same query."""
    lay = Layout(16, 576, 512)
    env = Located(dhs, lay, seed=17)
    loc = env.rand_loc(2, 90)
    it, t = env.item(loc)
    run(dhs, env.pool, lay, [it], q_strides=(576, 0))
    torch.cuda.synchronize()
    q = t[0].view(-1)[:2 * 576].view(2, 1, 576).expand(2, 16, 576)
    rows, keep = env.rows(loc)
    compare(lay, q, rows, keep, t[1], t[2])


def test_rows_past_4_gib(dhs):
    """An optional arena of 4.6 GB: rows whose byte offset passes 32 bits."""
    lay = LAYOUTS["latent"]
    pages = 4_100_000 // PAGE
    pool = dhs.Pool(max_requests=1, sources=1, row_bytes=1152, page_rows=PAGE, tail_rows=8,
                    hot_rows=8, max_queries=1, max_topk=8, max_rows_per_request=4096,
                    optional_pages=pages)
    opt = pool.opt.view(torch.bfloat16).view(-1, 576)
    last = torch.arange(4_100_000 - 300, 4_100_000 - 20, device="cuda")
    g = torch.Generator("cuda").manual_seed(1)
    opt[last] = torch.randn(len(last), 576, generator=g, device="cuda").bfloat16()
    loc = (last + (1 << 30))[None]
    lt = loc.to(torch.int32).contiguous()
    q = torch.randn(1, 16, 576, generator=g, device="cuda").bfloat16()
    out, lse = torch.empty(1, 16, 512, dtype=q.dtype, device="cuda"), torch.empty(1, 16, device="cuda")
    run(dhs, pool, lay, [dhs.attend_item(queries=1, topk=len(last), q=q, loc=lt, out=out, lse=lse)])
    torch.cuda.synchronize()
    compare(lay, q, opt[last][None], torch.ones(1, len(last), dtype=torch.bool, device="cuda"), out, lse)
    pool.close()


# ---------------------------------------------------------------- histories

class History:
    """One request per length, its rows known, half of the pages resident."""

    def __init__(self, dhs, lay, lens, T=24, window=False, appended=0, seed=0, resident=0.5,
                 stream=None):
        self.dhs, self.lay, self.lens, self.T, self.window = dhs, lay, lens, T, window
        self.g = torch.Generator("cuda").manual_seed(seed)
        n = max(lens) + appended + 1
        rb = lay.elems * 2
        self.rows = torch.randn(len(lens), n, lay.elems, generator=self.g, device="cuda").to(TYPES[lay.dtype])
        self.pool = dhs.Pool(max_requests=len(lens), sources=1, row_bytes=rb, page_rows=PAGE,
                             tail_rows=T, hot_rows=16, max_queries=8, max_topk=16,
                             max_rows_per_request=n, optional_pages=sum(x // PAGE for x in lens) + 1,
                             stream=stream)
        self.host = torch.zeros(len(lens), n * rb, dtype=torch.uint8).pin_memory()
        for r, x in enumerate(lens):
            if window:
                m = min(x, T)
                rc = self.pool.admit_window(r, 0, self.rows[r, x - m:].data_ptr(), x)
            else:
                mask = (torch.rand(x // PAGE, generator=self.g, device="cuda") < resident)
                rc = self.pool.admit_device(r, 0, self.rows[r].data_ptr(), self.host[r].data_ptr(), x,
                                            mask.cpu().numpy())[0]
            assert rc == 0
        step = 0
        while step < appended:  # decode rows, at most a ring at a time
            m = min(T, appended - step)
            items = []
            for r, x in enumerate(lens):
                a = dhs.dhs_append_item()
                a.req, a.count, a.rows_dev = r, m, self.rows[r, x + step].data_ptr()
                items.append(a)
            assert self.pool.append(items) == 0
            step += m
        self.len = [x + appended for x in lens]

    def items(self, Q, ranges=None):
        lay, out = self.lay, []
        for r in range(len(self.lens)):
            q = torch.randn(Q, lay.heads, lay.key, generator=self.g, device="cuda").to(TYPES[lay.dtype])
            o = torch.full((Q, lay.heads, lay.value), 7.0, dtype=q.dtype, device="cuda")
            lse = torch.full((Q, lay.heads), 7.0, device="cuda")
            rg = None if ranges is None else torch.tensor(ranges[r], dtype=torch.int32, device="cuda")
            it = self.dhs.attend_item(req=r, queries=Q, flags=self.dhs.DHS_ATTEND_HISTORY, q=q, out=o,
                                      lse=lse, range_=rg)
            out.append((it, (q, o, lse, rg)))
        return out

    def check(self, its, Q, ranges=None):
        torch.cuda.synchronize()
        for r, (_, (q, o, lse, _)) in enumerate(its):
            L = self.len[r]
            pos = torch.arange(L, device="cuda")
            lo = max(0, L - self.T) if self.window else 0
            keep = torch.stack([(pos >= max(lo, ranges[r][i][0] if ranges else 0)) &
                                (pos < (ranges[r][i][1] if ranges else L - Q + 1 + i))
                                for i in range(Q)])
            compare(self.lay, q, self.rows[r, :L][None], keep, o, lse)


@pytest.mark.parametrize("Q", [1, 4])
@pytest.mark.parametrize("name", ["latent", "latent_100", "grouped", "grouped_f16", "odd", "largest"])
def test_history(dhs, name, Q):
    """Rows in the ring, in pages that end inside a tile, and on the host;
    lengths from nothing to several tiles, decode rows past the import."""
    env = History(dhs, LAYOUTS[name], [0, 1, 2, 15, 16, 17, 127, 128, 129, 500], appended=0, seed=Q)
    its = env.items(Q)
    run(dhs, env.pool, env.lay, [i for i, _ in its])
    env.check(its, Q)
    env = History(dhs, LAYOUTS[name], [0, 3, 130, 411], appended=70, seed=Q)
    its = env.items(Q)
    run(dhs, env.pool, env.lay, [i for i, _ in its])
    env.check(its, Q)
    assert env.pool.status() == (0, 0)


@pytest.mark.parametrize("Q", [1, 3])
def test_history_window_source(dhs, Q):
    """A window source serves the last tail_rows rows, wherever its ring begins."""
    for T in (24, 200):
        env = History(dhs, LAYOUTS["latent"], [0, 1, 23, 24, 25, 199, 200, 333], T=T, window=True, seed=T)
        its = env.items(Q)
        run(dhs, env.pool, env.lay, [i for i, _ in its])
        env.check(its, Q)


def test_history_ranges(dhs):
    """Ranges of rows per query: empty, reversed, past both ends, one row."""
    lens = [300, 40, 0]
    ranges = [[[0, 300], [10, 11], [5, 5], [200, 100], [-50, 3], [299, 1000], [128, 256], [-5, -1]]] * 3
    for window in (False, True):
        env = History(dhs, LAYOUTS["grouped"], lens, T=24, window=window, seed=3)
        its = env.items(8, ranges)
        run(dhs, env.pool, env.lay, [i for i, _ in its])
        env.check(its, 8, ranges)


def test_history_fully_resident_and_long(dhs):
    """One 20000-row history, every page resident, split over the GPU."""
    for name in ("latent", "latent_64"):
        env = History(dhs, LAYOUTS[name], [20000], T=64, seed=1, resident=2.0)
        its = env.items(2)
        run(dhs, env.pool, env.lay, [i for i, _ in its])
        env.check(its, 2)


def test_history_many_queries_share_rows(dhs):
    """Q x heads beyond one block's columns, ragged against the block width."""
    env = History(dhs, Layout(20, 64, 64), [700], seed=2)
    its = env.items(8)
    run(dhs, env.pool, env.lay, [i for i, _ in its])
    env.check(its, 8)


def test_history_and_located_in_one_step(dhs):
    env = History(dhs, LAYOUTS["latent"], [260], seed=4, resident=2.0)
    its = env.items(2)
    # pages 0.. lie in slots 0..: row r is page row r of the optional arena
    loc = (torch.arange(64, device="cuda") + (1 << 30)).to(torch.int32)[None].contiguous()
    lay = env.lay
    q = torch.randn(1, lay.heads, lay.key, device="cuda").bfloat16()
    o, lse = torch.empty(1, lay.heads, lay.value, device="cuda").bfloat16(), torch.empty(1, lay.heads, device="cuda")
    run(dhs, env.pool, lay, [its[0][0], dhs.attend_item(queries=1, topk=64, q=q, loc=loc, out=o, lse=lse)])
    env.check(its, 2)
    compare(lay, q, env.rows[0, :64][None], torch.ones(1, 64, dtype=torch.bool, device="cuda"), o, lse)


# ------------------------------------------------------------------ streams

def test_attend_on_another_stream(dhs):
    """Ordered after the pool's work, and before its next change of rows."""
    lay = LAYOUTS["latent"]
    pool_stream, side = torch.cuda.Stream(), torch.cuda.Stream()
    with torch.cuda.stream(pool_stream):
        env = History(dhs, lay, [3000], T=24, seed=5, stream=pool_stream)
        its = env.items(1)
    torch.cuda.synchronize()
    old = env.rows[0].clone()
    # a busy pool stream: the append below must not overtake the attention
    rows = torch.randn(1, lay.elems, device="cuda").bfloat16()
    torch.cuda.synchronize()
    run(dhs, env.pool, lay, [its[0][0]], stream=side)
    a = dhs.dhs_append_item()
    a.count, a.rows_dev = 1, rows.data_ptr()
    assert env.pool.append([a]) == 0
    torch.cuda.synchronize()
    env.rows = old[None]
    env.check(its, 1)


# ----------------------------------------------------------------- refusals

def test_refusals(dhs):
    lay = LAYOUTS["latent"]
    env = Located(dhs, lay)
    loc = env.rand_loc(1, 10)
    E = dhs.DHS_EINVAL

    def attempt(item=(), step=(), work=True, **kw):
        it, t = env.item(loc)
        for k, v in dict(item).items():
            setattr(it, k, v)
        st, keep = dhs.make_attend([it], **{**lay.args(), **kw})
        for k, v in dict(step).items():
            setattr(st, k, v)
        buf = torch.empty(64 << 20, dtype=torch.uint8, device="cuda")
        if work:
            st.work_dev, st.work_bytes = buf.data_ptr(), buf.numel()
        rc = env.pool.attend(st)
        torch.cuda.synchronize()
        if rc:
            assert bool((t[1] == 7.0).all())
        return rc

    assert attempt() == 0
    for kw in (dict(heads=0), dict(kv_heads=0), dict(heads=5, kv_heads=2), dict(key_elems=584),
               dict(key_elems=0), dict(key_elems=12), dict(value_elems=520), dict(value_elems=4),
               dict(value_elems=-8), dict(key_offset=8), dict(value_offset=72), dict(value_offset=-8),
               dict(value_offset=4), dict(kv_heads=2, key_stride=8), dict(kv_heads=2, key_elems=64, key_stride=4),
               dict(kv_heads=2, key_elems=64, value_elems=64, key_stride=-64), dict(scale=float("inf")),
               dict(scale=NAN)):
        assert attempt(**kw) == E, kw
    assert attempt(step=dict(dtype=2)) == E
    assert attempt(step=dict(n_items=-1)) == E
    assert attempt(item=dict(queries=-1)) == E
    assert attempt(item=dict(topk=-1)) == E
    assert attempt(item=dict(flags=2)) == E
    assert attempt(item=dict(q_dev=None)) == E
    assert attempt(item=dict(out_dev=None)) == E
    assert attempt(item=dict(loc_dev=None)) == E
    assert attempt(item=dict(q_dev=loc.data_ptr() + 1)) == E
    assert attempt(item=dict(lse_dev=loc.data_ptr() + 2)) == E
    assert attempt(item=dict(flags=dhs.DHS_ATTEND_HISTORY, req=3)) == E
    assert attempt(item=dict(flags=dhs.DHS_ATTEND_HISTORY, src=-1)) == E
    assert attempt(item=dict(flags=dhs.DHS_ATTEND_HISTORY)) == dhs.DHS_ESTATE
    assert attempt(item=dict(queries=0, q_dev=None, out_dev=None)) == 0
    st, keep = dhs.make_attend([], **lay.args())
    assert env.pool.attend(st) == 0
    assert env.pool.attend_on(st, None) == E
    assert dhs.lib.dhs_attend_bytes(env.pool.h, None, None) == E
    # a workspace that is missing, short or misaligned
    big = env.rand_loc(1, 20000).to(torch.int32).contiguous()
    it, t = env.item(loc)
    it.loc_dev, it.topk = big.data_ptr(), 20000
    st, keep = dhs.make_attend([it], **lay.args())
    need = env.pool.attend_bytes(st)
    if need:
        buf = torch.empty(need + 256, dtype=torch.uint8, device="cuda")
        assert env.pool.attend(st) == E
        st.work_dev, st.work_bytes = buf.data_ptr(), need - 1
        assert env.pool.attend(st) == E
        st.work_dev, st.work_bytes = buf.data_ptr() + 16, need
        assert env.pool.attend(st) == E
        st.work_dev = buf.data_ptr()
        assert env.pool.attend(st) == 0
    torch.cuda.synchronize()


@pytest.mark.parametrize("name", ["latent", "latent_100", "grouped", "odd", "largest"])
@pytest.mark.parametrize("L", [3, 128, 130, 389])
def test_history_row_that_is_not_finite(dhs, name, L):
    """A row with NaN that only the block's later queries see leaves the
    earlier ones untouched."""
    lay, Q = LAYOUTS[name], 5
    env = History(dhs, lay, [L], T=24, seed=11)
    for back in (1, 2, 3):  # the last rows, the third from the end by query 2 on
        if L < back:
            continue
        rows = torch.full((1, lay.elems), NAN, device="cuda").to(env.rows.dtype)
        env.rows[0, L - back] = rows
    # a pool of its own whose ring holds the damaged rows
    pool = dhs.Pool(max_requests=1, sources=1, row_bytes=lay.elems * 2, page_rows=PAGE, tail_rows=24,
                    hot_rows=16, max_queries=8, max_topk=16, max_rows_per_request=L + 1,
                    optional_pages=L // PAGE + 1)
    host = torch.zeros((L + 1) * lay.elems * 2, dtype=torch.uint8).pin_memory()
    assert pool.admit_device(0, 0, env.rows[0].data_ptr(), host.data_ptr(), L)[0] == 0
    env.pool = pool
    (it, (q, o, lse, _)), = env.items(Q)
    run(dhs, pool, lay, [it])
    torch.cuda.synchronize()
    first_bad = max(0, L - 3)
    for i in range(Q):
        end = max(0, L - Q + 1 + i)
        if end > first_bad:
            assert bool(o[i].isnan().all()) and bool(lse[i].isnan().all()), i
        else:
            keep = torch.arange(L, device="cuda")[None] < end
            compare(lay, q[i:i + 1], env.rows[0, :L][None], keep, o[i:i + 1], lse[i:i + 1])


@pytest.mark.parametrize("name", ["grouped", "grouped_f16", "interleaved", "largest"])
def test_history_value_that_is_infinite(dhs, name):
    """An infinite value element reaches that element of the queries that see
    its row, and nothing else."""
    lay, Q, L = LAYOUTS[name], 4, 150
    env = History(dhs, lay, [L], T=24, seed=12, appended=0)
    g = lay.kv - 1
    at = lay.value_offset + g * lay.value_stride + 3
    clean = env.rows.clone()
    env.rows[0, L - 2, at] = math.inf
    pool = dhs.Pool(max_requests=1, sources=1, row_bytes=lay.elems * 2, page_rows=PAGE, tail_rows=24,
                    hot_rows=16, max_queries=8, max_topk=16, max_rows_per_request=L + 1,
                    optional_pages=L // PAGE + 1)
    host = torch.zeros((L + 1) * lay.elems * 2, dtype=torch.uint8).pin_memory()
    assert pool.admit_device(0, 0, env.rows[0].data_ptr(), host.data_ptr(), L)[0] == 0
    env.pool = pool
    (it, (q, o, lse, _)), = env.items(Q)
    run(dhs, pool, lay, [it])
    torch.cuda.synchronize()
    heads = slice(g * (lay.heads // lay.kv), lay.heads)
    sees = torch.arange(Q, device="cuda") >= 2  # rows below L - 3 + i include L - 2
    assert bool((o[sees][:, heads, 3] == math.inf).all())
    o[sees, heads, 3] = 0
    keep = torch.arange(L, device="cuda")[None] < (L - Q + 1 + torch.arange(Q, device="cuda"))[:, None]
    ro, rl, tol, ltol = reference(lay, q, clean[0, :L][None], keep)
    ro[sees, heads, 3] = 0
    assert bool(((o.double() - ro).abs() <= tol).all())
    assert bool(((lse.double() - rl).abs() <= ltol).all())
