"""dhs_attend_packed against the formula in 64 bits over what the rows' codes
stand for: located rows (all tiers, entries without a row, union lists) and
histories (ring, pages, host rows, windows), over head layouts, lengths, masks
and scales where a tiled, split kernel can go wrong.

Bounds, from the number formats alone.  With weights w_j summing to 1, values
y_j = 2^v_j d_j and A = sum w_j |y_j|:
  - weights: bf16 three e5m2 pieces of a number rounded to f16, 2^-9 + 2^-11 of
    each; f16 2^-11; each at least to half of e5m2's smallest number, 2^-17,
    where the largest 2^v_j w_j is at least 2^9 (the reference's height):
    multiplied by a code F = 2^-26 max_j(2^v_j w_j) sum_j |d_j|;
  - queries: to 2^-18 of the largest coded element, a score by at most
    q = 2^-18 max|a| scale sum_e |key_je|;
  - scores: float accumulation of key elements in steps of at least 16, with the
    sums of pieces, d = 2^-22 (key / 16 + 8) max_j scale sum |q x_j|;
  - sums over n rows in steps of 32: 2^-23 (n / 32 + 8) A;
  - the output's own rounding, u |out|.
An error d + q of the scores moves the output by 2 (d + q) A, the log-sum by
d + q and the roundings of its own logarithm and sum.
"""
import math

import pytest
import torch

from packed_layouts import LAYOUTS, Layout

pytestmark = pytest.mark.gpu

U = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11}
W = {"bf16": 2.0 ** -9 + 2.0 ** -11, "f16": 2.0 ** -11}
PAGE = 16
NAN_CODE = 0x7F


@pytest.fixture(scope="module")
def dhs():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from hierarchical_sparse_kv_dhs_gb300.build import build
    build()
    from hierarchical_sparse_kv_dhs_gb300 import dhs as mod
    return mod


def reference(lay, q, rows, keep):
    """Outputs and bounds in 64 bits: q [Q, H, dk], rows [Q or 1, n, bytes], keep [Q, n]."""
    Q, H = q.shape[:2]
    share, u = H // lay.kv, U[lay.dtype]
    out = torch.zeros(Q, H, lay.value, dtype=torch.float64, device=q.device)
    lse = torch.full((Q, H), -math.inf, dtype=torch.float64, device=q.device)
    tol, ltol = torch.zeros_like(out), torch.zeros_like(lse)
    for i in range(Q):
        r = rows[i if rows.shape[0] > 1 else 0][keep[i]]
        n = len(r)
        if n == 0:
            continue
        keys, values = lay.numbers(r)
        scales = r[:, lay.off_scale:lay.off_scale + 4 * lay.scales].contiguous().view(torch.float32)
        for g in range(lay.kv):
            hs = slice(g * share, (g + 1) * share)
            x, y, qg = keys[:, g], values[:, g], q[i, hs].double()
            s = qg @ x.T * lay.scale
            m = s.amax(1, keepdim=True)
            p = torch.exp(s - m.masked_fill(m == -math.inf, 0))
            z = p.sum(1, keepdim=True)
            w = p / z.masked_fill(z == 0, 1)
            out[i, hs], lse[i, hs] = w @ y, (m + torch.log(z))[:, 0]
            big = (qg.abs() @ x.abs().T).amax(1, keepdim=True) * lay.scale
            d = 2.0 ** -22 * (lay.key / 16 + 8) * big
            top = qg[:, :lay.key8].abs().amax(1, keepdim=True)
            d = d + 2.0 ** -18 * top * lay.scale * x[:, :lay.key8].abs().sum(1).amax()
            vs = scales[:, g if lay.shared else lay.kv + g].double()
            floor = 2.0 ** -26 * (w * vs).amax(1, keepdim=True) * (y / vs[:, None]).abs().sum(0)
            a = w @ y.abs()
            tol[i, hs] = (1.02 * W[lay.dtype] + 2 * d + 2.0 ** -23 * (n / 32 + 8)) * a + \
                1.02 * u * out[i, hs].abs() + floor + 2.0 ** -25
            ltol[i, hs] = d[:, 0] + 2.0 ** -21 * (lse[i, hs].abs() + 1)
    return out, lse, tol, ltol


def compare(lay, q, rows, keep, out, lse):
    ro, rl, tol, ltol = reference(lay, q, rows, keep)
    # A number from finfo.max plus half a unit on rounds to infinity (the tests'
    # value scales go up to 2^30, an f16's numbers to 65504 < 2^16).
    top = torch.finfo(lay.type).max * (1 + U[lay.dtype] / 2)
    past = ro.abs() - tol >= top
    assert torch.equal(out[past].double(), ro[past].sign() * math.inf)
    near = ~past & (ro.abs() + tol >= top)  # either is right
    err = (out.double() - ro).abs().masked_fill(past | (near & out.isinf()), 0)
    assert bool((err <= tol).all()), f"output off by {(err / tol.clamp(min=1e-300)).max():.3g} bounds"
    none = rl == -math.inf
    assert torch.equal(none, lse == -math.inf)
    assert bool((out[none] == 0).all())
    e = (lse.double() - rl).abs()
    assert bool((e[~none] <= ltol[~none]).all()), f"log-sum off by {(e / ltol)[~none].max():.3g} bounds"


def step_of(dhs, pool, lay, items, **kw):
    st, keep = dhs.make_attend_packed(items, lay.rows(dhs), **{**dict(heads=lay.heads, scale=lay.scale), **kw})
    work = torch.empty(max(256, pool.attend_packed_bytes(st)), dtype=torch.uint8, device="cuda").fill_(0xA5)
    st.work_dev, st.work_bytes = work.data_ptr(), work.numel()
    return st, (keep, work)


def run(dhs, pool, lay, items, stream=None, **kw):
    st, keep = step_of(dhs, pool, lay, items, **kw)
    rc = pool.attend_packed_on(st, stream.cuda_stream) if stream else pool.attend_packed(st)
    assert rc == 0, dhs.lib.dhs_strerror(rc)
    return keep


class Located:
    """A pool with caller-given arenas of random rows, and location vectors."""

    def __init__(self, dhs, lay, R=3, T=20, B=50, pages=30, seed=0):
        self.dhs, self.lay = dhs, lay
        self.g = torch.Generator("cuda").manual_seed(seed)
        self.sizes = [R * B, R * T, pages * PAGE]  # hot, tail, opt
        self.arenas = [lay.random(n, self.g) for n in self.sizes]
        self.pool = dhs.Pool(max_requests=R, sources=1, row_bytes=lay.row_bytes, page_rows=PAGE,
                             tail_rows=T, hot_rows=B, max_queries=8, max_topk=64,
                             max_rows_per_request=4096, optional_pages=pages,
                             arenas=[a.view(-1) for a in self.arenas])

    def rand_loc(self, Q, k):
        hot, tail, opt = self.sizes
        tier = torch.randint(0, 3, (Q, k), generator=self.g, device="cuda")
        n = torch.tensor([tail, opt, hot], device="cuda")[tier]
        return (tier << 30) + (torch.rand(Q, k, generator=self.g, device="cuda") * n).long()

    def distinct(self, k):
        """k locations of different rows."""
        hot, tail, opt = self.sizes
        x = torch.randperm(hot + tail + opt, generator=self.g, device="cuda")[:k]
        return torch.where(x < tail, x, torch.where(x < tail + opt, x - tail + (1 << 30),
                                                    x - tail - opt + (2 << 30)))[None]

    def rows(self, loc):
        keep = loc < 0xC0000000
        tier, x = torch.where(keep, loc >> 30, 0), torch.where(keep, loc & 0x3FFFFFFF, 0)
        hot, tail, opt = self.arenas
        first = torch.tensor([0, len(tail), len(tail) + len(opt)], device="cuda")
        return torch.cat([tail, opt, hot])[first[tier] + x], keep

    def write(self, loc, rows):
        """Rows [k, bytes] at loc [1, k]."""
        for t, a in zip((2, 0, 1), self.arenas):
            at = (loc[0] >> 30) == t
            a[loc[0][at] & 0x3FFFFFFF] = rows[at]

    def poison(self, loc):
        """NaN codes, elements and scales in every row that no location names."""
        for t, a in zip((2, 0, 1), self.arenas):
            named = torch.zeros(len(a), dtype=torch.bool, device="cuda")
            named[(loc[(loc < 0xC0000000) & (loc >> 30 == t)] & 0x3FFFFFFF)] = True
            a[~named] = 0xFF

    def item(self, loc, index=None):
        Q, k = loc.shape
        lay = self.lay
        q = torch.randn(Q, lay.heads, lay.key, generator=self.g, device="cuda").to(lay.type)
        out = torch.full((Q, lay.heads, lay.value), 7.0, dtype=q.dtype, device="cuda")
        lse = torch.full((Q, lay.heads), 7.0, device="cuda")
        keep = loc.to(torch.int32).contiguous()
        it = self.dhs.attend_item(queries=Q, topk=k, q=q, loc=keep, index=index, out=out, lse=lse)
        return it, (q, out, lse, keep)


def check_located(env, cases):
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


@pytest.mark.parametrize("name", ["latent", "latent_64", "grouped_f16", "odd", "no_wide_64"])
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


@pytest.mark.parametrize("name", ["latent", "latent_f16", "latent_128", "grouped", "no_wide_f16"])
def test_located_long_selection_split_over_blocks(dhs, name):
    """One query over 5000 entries (duplicates included) is split and joined;
    the same call twice gives the same bits."""
    env = Located(dhs, LAYOUTS[name], seed=9)
    loc = env.rand_loc(1, 5000)
    it, t = env.item(loc)
    run(dhs, env.pool, env.lay, [it])
    check_located(env, [(loc, t)])
    first = t[1].clone(), t[2].clone()
    run(dhs, env.pool, env.lay, [it])
    torch.cuda.synchronize()
    assert torch.equal(first[0], t[1]) and torch.equal(first[1], t[2])


@pytest.mark.parametrize("name", ["latent", "odd", "grouped_wide"])
@pytest.mark.parametrize("items", [1, 17, 250])
def test_located_ragged_items(dhs, name, items):
    """Items of different Q and k in one step, more than one launch table and
    more segments a block than are found ahead."""
    env = Located(dhs, LAYOUTS[name], seed=items)
    cases, its = [], []
    for i in range(items):
        loc = env.rand_loc(i % 4, (37 * i) % 290)
        it, t = env.item(loc)
        its.append(it)
        cases.append((loc, t))
    run(dhs, env.pool, env.lay, its)
    check_located(env, [c for c in cases if c[0].shape[0]])


@pytest.mark.parametrize("name", ["latent", "latent_64", "grouped"])
def test_located_waves_of_equal_jobs(dhs, name):
    """Many equal jobs: several whole ones a block, the queries of the next
    loaded behind those of the one before."""
    env = Located(dhs, LAYOUTS[name], seed=1)
    cases, its = [], []
    for i in range(80):
        loc = env.rand_loc(8, 290)
        it, t = env.item(loc)
        its.append(it)
        cases.append((loc, t))
    run(dhs, env.pool, env.lay, its)
    check_located(env, cases[::13])
    assert env.pool.status() == (0, 0)


def test_located_union_index(dhs):
    """A union list with per-query positions; negative positions are no row,
    positions past the list raise ELOC."""
    env = Located(dhs, LAYOUTS["latent"], seed=3)
    Q, k, n = 4, 150, 200
    lst = env.rand_loc(1, Q * k).view(Q, k)
    flat = lst.view(-1)
    flat[n:] = 0xFFFFFFFE
    index = torch.randint(0, n, (Q, k), generator=env.g, device="cuda")
    index[torch.rand(Q, k, generator=env.g, device="cuda") < 0.2] = -1
    index[2] = -1
    idx32 = index.to(torch.int32)
    it, t = env.item(lst, index=idx32)
    run(dhs, env.pool, env.lay, [it])
    seen = torch.where(index >= 0, flat[index.clamp(min=0)], 0xFFFFFFFF)
    check_located(env, [(seen, t)])
    idx32[0, 0] = Q * k
    seen[0, 0] = 0xFFFFFFFF
    run(dhs, env.pool, env.lay, [it])
    check_located(env, [(seen, t)])
    assert env.pool.status() == (dhs.DHS_ERANGE, dhs.DHS_STATUS_ELOC)


def test_located_out_of_arena(dhs):
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


def directed(env, loc, t, scores, value_exp=None):
    """Distinct rows at loc [1, k] whose scores are scores[j] for every head
    (coded: 64 * 2^e and a part in a second element), and value scales."""
    lay, k = env.lay, loc.shape[1]
    q = t[0]
    q.zero_()
    q[..., 0], q[..., 1] = 1.0, 1.0 / 16
    n = lay.random(k, env.g)
    key = n[:, :lay.off_value].view(k, lay.kv, -1)
    # scores in multiples of 1/16 of the step below: (a + b / 16) 2^e
    want = scores.double() / lay.scale
    e = torch.ceil(torch.log2(want.abs().clamp(min=2.0 ** -20) / 448))
    a = (want / torch.exp2(e)).float().to(torch.float8_e4m3fn)
    b = ((want / torch.exp2(e) - a.double()) * 16).float().to(torch.float8_e4m3fn)
    key[..., 0], key[..., 1] = a.view(torch.uint8)[:, None], b.view(torch.uint8)[:, None]
    scale = n[:, lay.off_scale:lay.off_scale + 4 * lay.scales].contiguous().view(torch.float32)
    scale[:, :lay.kv] = torch.exp2(e).float()[:, None]
    if value_exp is not None and not lay.shared:
        scale[:, lay.kv:] = torch.exp2(value_exp.float())[:, None]
    n[:, lay.off_scale:lay.off_scale + 4 * lay.scales] = scale.view(torch.uint8).view(k, -1)
    if lay.wide:
        n[:, lay.off_wide:lay.off_scale] = 0
    env.write(loc, n)


@pytest.mark.parametrize("name", ["latent", "latent_64", "grouped", "grouped_f16", "no_wide_64"])
@pytest.mark.parametrize("shape", ["rising", "falling", "spike", "wide", "flat"])
def test_located_score_ranges(dhs, name, shape):
    """Scores whose maximum moves all the time, or by much more than exp's range."""
    env = Located(dhs, LAYOUTS[name], B=200, seed=6)
    k = 600
    n = torch.arange(k, device="cuda", dtype=torch.float32)
    scores = {"rising": n / 4 - 70, "falling": 70 - n / 4, "spike": torch.where(n == 401, 300.0, -300.0),
              "wide": (n * 37 % k) - 300, "flat": torch.zeros(k, device="cuda")}[shape]
    loc = env.distinct(k)
    it, t = env.item(loc)
    directed(env, loc, t, scores)
    run(dhs, env.pool, env.lay, [it])
    check_located(env, [(loc, t)])


@pytest.mark.parametrize("name", ["grouped", "grouped_f16", "no_wide_64"])
@pytest.mark.parametrize("shape", ["small_at_top", "large_at_top", "spread"])
def test_located_value_scales(dhs, name, shape):
    """Value scales far apart, with the scores or against them: a row that takes
    the weight but hardly a value, and the other way round."""
    env = Located(dhs, LAYOUTS[name], B=200, seed=7)
    k = 500
    n = torch.arange(k, device="cuda", dtype=torch.float32)
    top = n == 300
    scores = torch.where(top, 12.0, 0.0) if shape != "spread" else (n * 29 % 97) / 12
    exps = {"small_at_top": torch.where(top, -64, 3), "large_at_top": torch.where(top, 30, -20),
            "spread": (n * 17 % 61).long() - 30}[shape]
    loc = env.distinct(k)
    it, t = env.item(loc)
    directed(env, loc, t, scores, exps)
    run(dhs, env.pool, env.lay, [it])
    check_located(env, [(loc, t)])


@pytest.mark.parametrize("name", ["latent_one_head", "grouped_f16"])
def test_one_row_that_stands_out(dhs, name):
    """A row with half of the weight beside 200000 that share the other half:
    weights 2^-18 of the largest count."""
    env = Located(dhs, LAYOUTS[name], B=200, seed=8)
    lay, k = env.lay, 200001
    one = env.distinct(65)
    it, t = env.item(one)
    directed(env, one, t, torch.cat([torch.tensor([math.log(200000.0)], device="cuda"),
                                     torch.zeros(64, device="cuda")]))
    loc = one[0, 1:][torch.arange(k, device="cuda") % 64][None].clone()
    loc[0, 77777] = one[0, 0]
    it2, t2 = env.item(loc)
    t2[0].copy_(t[0])
    run(dhs, env.pool, lay, [it2])
    check_located(env, [(loc, t2)])


def test_query_that_is_not_finite(dhs):
    """NaN for a query with NaN or an infinity among its coded elements; the
    others are untouched.  Zero queries weigh all rows alike."""
    for name in ("latent", "grouped_f16"):
        env = Located(dhs, LAYOUTS[name], seed=2)
        loc = env.rand_loc(4, 200)
        it, t = env.item(loc)
        t[0][1, 0, 3] = math.nan
        t[0][2, 1, 0] = math.inf
        t[0][3] = 0
        run(dhs, env.pool, env.lay, [it])
        torch.cuda.synchronize()
        for i, h in ((1, 0), (2, 1)):
            assert bool(t[1][i, h].isnan().all()) and bool(t[2][i, h].isnan())
            t[1][i, h], t[2][i, h], t[0][i, h] = 0, 0, 0
        rows, keep = env.rows(loc)
        ro, rl, tol, ltol = reference(env.lay, t[0], rows, keep)
        ro[1, 0], rl[1, 0], ro[2, 1], rl[2, 1] = 0, 0, 0, 0
        assert bool(((t[1].double() - ro).abs() <= tol).all())
        assert bool(((t[2].double() - rl).abs() <= ltol).all())


@pytest.mark.parametrize("size", [2.0 ** -30, 2.0 ** -14, 1.0, 2.0 ** 10])
@pytest.mark.parametrize("name", ["latent", "grouped_f16"])
def test_query_sizes(dhs, name, size):
    """Queries far from 1, with elements 2^-12 of the largest that count."""
    lay = LAYOUTS[name]
    if lay.dtype == "f16" and size < 2.0 ** -14:
        size = 2.0 ** -20  # subnormal
    env = Located(dhs, Layout(lay.heads, lay.key, lay.value, lay.kv, lay.wide, lay.shared, lay.dtype), seed=3)
    env.lay.scale = lay.scale / size
    loc = env.rand_loc(2, 150)
    it, t = env.item(loc)
    t[0].mul_(size)
    t[0][..., 1::2] *= 2.0 ** -12 if lay.dtype == "bf16" else 1
    run(dhs, env.pool, env.lay, [it])
    check_located(env, [(loc, t)])


def test_strides_alignment_and_missing_log_sum(dhs):
    """Queries and outputs as [H][Q] slices of wider, misaligned buffers;
    nothing outside the outputs is written."""
    for name in ("grouped", "latent"):
        lay = LAYOUTS[name]
        env = Located(dhs, lay, seed=7)
        Q, k = 3, 70
        loc = env.rand_loc(Q, k)
        lt = loc.to(torch.int32).contiguous()
        a, b = lay.key + 22, lay.value + 12
        for off in (0, 1, 5):
            qb = torch.randn(lay.heads * Q * a + 8, generator=env.g, device="cuda").to(lay.type)
            ob = torch.full((lay.heads * Q * b + 8,), 3.0, device="cuda").to(lay.type)
            q = torch.as_strided(qb, (Q, lay.heads, lay.key), (a, Q * a, 1), off)
            o = torch.as_strided(ob, (Q, lay.heads, lay.value), (b, Q * b, 1), off)
            it = dhs.attend_item(queries=Q, topk=k, q=qb.data_ptr() + 2 * off, loc=lt,
                                 out=ob.data_ptr() + 2 * off)
            run(dhs, env.pool, lay, [it], q_strides=(a, Q * a), out_strides=(b, Q * b))
            torch.cuda.synchronize()
            rows, keep = env.rows(loc)
            ro, rl, tol, _ = reference(lay, q, rows, keep)
            assert bool(((o.double() - ro).abs() <= tol).all())
            o.fill_(3.0)
            assert bool((ob == 3.0).all())


def test_rows_past_4_gib(dhs):
    """An optional arena of 4.6 GB: rows whose byte offset passes 32 bits."""
    lay = LAYOUTS["latent"]
    n = 7_000_000
    pool = dhs.Pool(max_requests=1, sources=1, row_bytes=lay.row_bytes, page_rows=PAGE, tail_rows=8,
                    hot_rows=8, max_queries=1, max_topk=8, max_rows_per_request=4096,
                    optional_pages=n // PAGE)
    opt = pool.opt.view(-1, lay.row_bytes)
    last = torch.arange(n - 300, n - 20, device="cuda")
    g = torch.Generator("cuda").manual_seed(1)
    opt[last] = lay.random(len(last), g)
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

    def __init__(self, dhs, lay, lens, T=24, window=False, seed=0, resident=0.5, stream=None,
                 change=None):
        self.dhs, self.lay, self.len, self.T, self.window = dhs, lay, lens, T, window
        self.g = torch.Generator("cuda").manual_seed(seed)
        n = max(lens) + 1
        self.rows = torch.stack([lay.random(n, self.g) for _ in lens])
        if change:
            change(self.rows)
        self.pool = dhs.Pool(max_requests=len(lens), sources=1, row_bytes=lay.row_bytes,
                             page_rows=PAGE, tail_rows=T, hot_rows=16, max_queries=8, max_topk=16,
                             max_rows_per_request=n + 8, stream=stream,
                             optional_pages=sum(x // PAGE for x in lens) + 1)
        self.host = torch.zeros(len(lens), (n + 8) * lay.row_bytes, dtype=torch.uint8).pin_memory()
        for r, x in enumerate(lens):
            if window:
                m = min(x, T)
                rc = self.pool.admit_window(r, 0, self.rows[r, x - m:].data_ptr(), x)
            else:
                mask = (torch.rand(x // PAGE, generator=self.g, device="cuda") < resident)
                rc = self.pool.admit_device(r, 0, self.rows[r].data_ptr(), self.host[r].data_ptr(), x,
                                            mask.cpu().numpy())[0]
            assert rc == 0

    def items(self, Q, ranges=None):
        lay, out = self.lay, []
        for r in range(len(self.len)):
            q = torch.randn(Q, lay.heads, lay.key, generator=self.g, device="cuda").to(lay.type)
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
@pytest.mark.parametrize("name", ["latent", "latent_100", "latent_64_f16", "grouped", "grouped_wide",
                                  "grouped_some_wide", "odd", "no_wide", "part_of_key"])
def test_history(dhs, name, Q):
    """Rows in the ring, in pages that end inside a tile, and on the host;
    lengths from nothing to several tiles."""
    env = History(dhs, LAYOUTS[name], [0, 1, 2, 15, 16, 17, 127, 128, 129, 500], seed=Q)
    its = env.items(Q)
    run(dhs, env.pool, env.lay, [i for i, _ in its])
    env.check(its, Q)
    assert env.pool.status() == (0, 0)


@pytest.mark.parametrize("Q", [1, 3])
@pytest.mark.parametrize("T", [24, 200])
def test_history_window_source(dhs, Q, T):
    env = History(dhs, LAYOUTS["latent"], [0, 1, 23, 24, 25, 199, 200, 333], T=T, window=True, seed=T)
    its = env.items(Q)
    run(dhs, env.pool, env.lay, [i for i, _ in its])
    env.check(its, Q)


@pytest.mark.parametrize("window", [False, True])
@pytest.mark.parametrize("name", ["grouped", "latent"])
def test_history_ranges(dhs, name, window):
    """Ranges of rows per query: empty, reversed, past both ends, one row."""
    ranges = [[[0, 300], [10, 11], [5, 5], [200, 100], [-50, 3], [299, 1000], [128, 256], [-5, -1]]] * 3
    env = History(dhs, LAYOUTS[name], [300, 40, 0], window=window, seed=3)
    its = env.items(8, ranges)
    run(dhs, env.pool, env.lay, [i for i, _ in its])
    env.check(its, 8, ranges)


@pytest.mark.parametrize("name", ["latent", "latent_64", "no_wide_64", "grouped"])
def test_history_fully_resident_and_long(dhs, name):
    """One 20000-row history, every page resident, split over the GPU."""
    env = History(dhs, LAYOUTS[name], [20000], T=64, seed=1, resident=2.0)
    its = env.items(2)
    run(dhs, env.pool, env.lay, [i for i, _ in its])
    env.check(its, 2)


@pytest.mark.parametrize("name", ["latent", "latent_100", "grouped", "odd", "no_wide", "part_of_key"])
@pytest.mark.parametrize("L", [3, 128, 130, 389])
def test_history_row_that_is_not_a_number(dhs, name, L):
    """NaN in a row that only the block's later queries see leaves the earlier
    ones untouched: in every element, or in one of the value."""
    lay, Q = LAYOUTS[name], 5

    def every(rows):
        rows[0, L - 2:L] = NAN_CODE

    env = History(dhs, lay, [L], seed=11, change=every)
    (it, (q, o, lse, _)), = env.items(Q)
    run(dhs, env.pool, lay, [it])
    torch.cuda.synchronize()
    for i in range(Q):
        end = max(0, L - Q + 1 + i)
        if end > L - 2:
            assert bool(o[i].isnan().all()) and bool(lse[i].isnan().all()), i
        else:
            keep = torch.arange(L, device="cuda")[None] < end
            compare(lay, q[i:i + 1], env.rows[0, :L][None], keep, o[i:i + 1], lse[i:i + 1])
    if lay.shared:
        return
    g = lay.kv - 1
    at = lay.off_value + g * lay.value + 3
    clean = []

    def one(rows):
        clean.append(rows.clone())
        rows[0, L - 2, at] = NAN_CODE | 0x80

    env = History(dhs, lay, [L], seed=12, change=one)
    (it, (q, o, lse, _)), = env.items(Q)
    run(dhs, env.pool, lay, [it])
    torch.cuda.synchronize()
    heads = slice(g * (lay.heads // lay.kv), lay.heads)
    sees = L - Q + 1 + torch.arange(Q, device="cuda") > L - 2
    assert bool(o[sees][:, heads, 3].isnan().all())
    o[sees, heads, 3] = 0
    keep = torch.arange(L, device="cuda")[None] < (L - Q + 1 + torch.arange(Q, device="cuda"))[:, None]
    ro, rl, tol, ltol = reference(lay, q, clean[0][0, :L][None], keep)
    ro[sees, heads, 3] = 0
    assert bool(((o.double() - ro).abs() <= tol).all())
    none = rl == -math.inf
    assert bool(((lse.double() - rl).abs() <= ltol)[~none].all()) and bool((lse[none] == -math.inf).all())


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

@pytest.mark.parametrize("name", ["latent", "latent_128", "grouped"])
def test_captured_and_replayed(dhs, name):
    """Replays with other queries and rows at the same addresses."""
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        lay = LAYOUTS[name]
        env = Located(dhs, lay, seed=1)
        loc = env.rand_loc(2, 3000)
        it, t = env.item(loc)
        st, keep = step_of(dhs, env.pool, lay, [it])
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        graph.capture_begin()
        assert env.pool.stream == side and env.pool.attend_packed(st) == 0
        graph.capture_end()
        for _ in range(2):
            t[0].normal_(generator=env.g)
            for a in env.arenas:
                a.copy_(lay.random(len(a), env.g))
            t[1].zero_()
            graph.replay()
            check_located(env, [(loc, t)])
    assert env.pool.status() == (0, 0)


def test_two_streams_at_once(dhs):
    """Two attentions on streams of their own, a workspace each."""
    lay = LAYOUTS["latent"]
    env = Located(dhs, lay, seed=13)
    jobs = []
    for _ in range(2):
        loc = env.rand_loc(1, 6000)
        it, t = env.item(loc)
        jobs.append((loc, it, t, torch.cuda.Stream()))
    torch.cuda.synchronize()
    keep = []
    for _ in range(5):
        for loc, it, t, stream in jobs:
            keep.append(run(dhs, env.pool, lay, [it], stream=stream))
    check_located(env, [(loc, t) for loc, _, t, _ in jobs])
    assert env.pool.status() == (0, 0)


@pytest.mark.parametrize("polls", [0, 1, 7])
@pytest.mark.parametrize("name", ["latent", "latent_128", "grouped", "no_wide"])
def test_waits_that_run_out(dhs, name, polls):
    """A launch that gives up ends, says so and leaves the pool usable."""
    env = Located(dhs, LAYOUTS[name], seed=polls)
    cases, items = [], []
    for Q, k in [(1, 2500)] + [(8, 130)] * 30 + [(8, 0)] * 40:
        loc = env.rand_loc(Q, k)
        it, t = env.item(loc)
        items.append(it)
        cases.append((loc, t))
    env.pool.set_option(dhs.DHS_OPT_ATTEND_POLLS, polls)
    late = (dhs.DHS_ETIMEDOUT, dhs.DHS_STATUS_ETIMEDOUT)
    for _ in range(3):
        run(dhs, env.pool, env.lay, items)
        status = env.pool.status()
        assert status == late if polls == 0 else status in (late, (0, 0))
    env.pool.set_option(dhs.DHS_OPT_ATTEND_POLLS, -1)
    run(dhs, env.pool, env.lay, items)
    check_located(env, cases)
    assert env.pool.status() == (0, 0)


# ----------------------------------------------------------------- refusals

def test_refusals(dhs):
    lay = LAYOUTS["latent"]
    env = Located(dhs, lay)
    loc = env.rand_loc(1, 10)
    E = dhs.DHS_EINVAL

    def attempt(item=(), step=(), rows=(), **kw):
        it, t = env.item(loc)
        for k, v in dict(item).items():
            setattr(it, k, v)
        st, keep = dhs.make_attend_packed([it], lay.rows(dhs), **{**dict(heads=16, scale=0.1), **kw})
        for k, v in dict(step).items():
            setattr(st, k, v)
        for k, v in dict(rows).items():
            setattr(st.rows, k, v)
        buf = torch.empty(1 << 20, dtype=torch.uint8, device="cuda")
        st.work_dev, st.work_bytes = buf.data_ptr(), buf.numel()
        rc = env.pool.attend_packed(st)
        torch.cuda.synchronize()
        if rc:
            assert bool((t[1] == 7.0).all())
        return rc

    assert attempt() == 0
    for rows in (dict(dtype=2), dict(kv_heads=0), dict(kv_heads=2), dict(key_elems=592), dict(key_elems=560),
                 dict(wide_elems=72), dict(wide_elems=60), dict(wide_elems=-8), dict(value_elems=528),
                 dict(value_elems=0), dict(value_elems=24), dict(shared=2), dict(shared=0)):
        assert attempt(rows=rows) == E, rows
    assert attempt(heads=0) == E and attempt(scale=math.inf) == E and attempt(scale=math.nan) == E
    assert attempt(step=dict(n_items=-1)) == E
    for item in (dict(queries=-1), dict(topk=-1), dict(flags=2), dict(q_dev=None), dict(out_dev=None),
                 dict(loc_dev=None), dict(q_dev=loc.data_ptr() + 1), dict(lse_dev=loc.data_ptr() + 2),
                 dict(flags=dhs.DHS_ATTEND_HISTORY, req=3), dict(flags=dhs.DHS_ATTEND_HISTORY, src=-1)):
        assert attempt(item=item) == E, item
    assert attempt(item=dict(flags=dhs.DHS_ATTEND_HISTORY)) == dhs.DHS_ESTATE
    assert attempt(item=dict(queries=0, q_dev=None, out_dev=None)) == 0
    st, keep = dhs.make_attend_packed([], lay.rows(dhs), heads=16, scale=1.0)
    assert env.pool.attend_packed(st) == 0
    assert env.pool.attend_packed_on(st, None) == E
    assert dhs.lib.dhs_attend_packed_bytes(env.pool.h, None, None) == E
    # a workspace that is missing, short or misaligned
    big = env.rand_loc(1, 20000).to(torch.int32).contiguous()
    it, t = env.item(loc)
    it.loc_dev, it.topk = big.data_ptr(), 20000
    st, keep = dhs.make_attend_packed([it], lay.rows(dhs), heads=16, scale=0.1)
    need = env.pool.attend_packed_bytes(st)
    assert need > 0
    buf = torch.empty(need + 256, dtype=torch.uint8, device="cuda")
    assert env.pool.attend_packed(st) == E
    st.work_dev, st.work_bytes = buf.data_ptr(), need - 1
    assert env.pool.attend_packed(st) == E
    st.work_dev, st.work_bytes = buf.data_ptr() + 16, need
    assert env.pool.attend_packed(st) == E
    st.work_dev = buf.data_ptr()
    assert env.pool.attend_packed(st) == 0
    torch.cuda.synchronize()
