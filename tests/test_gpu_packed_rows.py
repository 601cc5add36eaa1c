"""Rotary positions, packed rows and reading them back, against plain forms in
64 bits.

Bounds.  A rotation's angle is a fraction of a turn held to 2^-32 and reduced to
a float of at most an eighth of a turn: off by at most 2 pi (2^-32 + 2^-27) <
2^-24; sine and cosine by 2^-23 with that, times the amplitude another 2^-24;
two products and a sum 2^-23 of |a| + |b|: 2^-21 (|a| + |b|) amplitude in all,
then one rounding, u of the result (2^-8 bf16, 2^-11 f16).  The table: a double
f / (2 pi) 2^64, a few 2^-53 of it, at 2^31 positions under 2^-20 of a turn.

A code is off by half a step of 2^-3 of its power of two: a rotation's error e
can move an element to the neighbouring code, so that the number differs from
the rule's for the exact element by at most one step more, and only where the
exact element lies within e of a border between codes; the scale likewise where
the largest element lies within e of 448 times a power of two.
"""
import math

import pytest
import torch

from packed_layouts import LAYOUTS, Layout, TYPES, codes_of

pytestmark = pytest.mark.gpu

U = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11}
PAGE = 16


@pytest.fixture(scope="module")
def dhs():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from hierarchical_sparse_kv_dhs_gb300.build import build
    build()
    from hierarchical_sparse_kv_dhs_gb300 import dhs as mod
    return mod


def pool_of(dhs, row_bytes=16, **kw):
    args = dict(max_requests=1, sources=1, row_bytes=row_bytes, page_rows=PAGE, tail_rows=8, hot_rows=16,
                max_queries=1, max_topk=16, max_rows_per_request=64, optional_pages=0)
    return dhs.Pool(**{**args, **kw})


def frequencies(n, base=10000.0, scaling="plain", factor=1.0, original=0.0, fast=32.0, slow=1.0):
    if scaling == "base":
        base *= factor ** (n / (n - 2))
    f = torch.tensor([base ** (-2.0 * i / n) for i in range(n // 2)], dtype=torch.float64)
    if scaling == "linear":
        f = f / factor
    if scaling == "parts":
        keep = ((original * f / (2 * math.pi) - slow) / (fast - slow)).clamp(0, 1)
        f = f * keep + f / factor * (1 - keep)
    return f


def turned(x, positions, f, pairs, amplitude=1.0, inverse=False):
    """x [n, heads, rotary] in 64 bits, and |a| + |b| of each element's pair."""
    t = positions.double()[:, None] * f.to(x.device)
    t = t[:, None] * (-1 if inverse else 1)
    c, s = torch.cos(t) * amplitude, torch.sin(t) * amplitude
    x = x.double()
    if pairs == "half":
        a, b = x.chunk(2, -1)
        m = a.abs() + b.abs()
        return torch.cat([a * c - b * s, b * c + a * s], -1), torch.cat([m, m], -1)
    a, b = x[..., 0::2], x[..., 1::2]
    m = a.abs() + b.abs()
    return torch.stack([a * c - b * s, b * c + a * s], -1).flatten(-2), torch.stack([m, m], -1).flatten(-2)


SCALINGS = [dict(), dict(scaling="linear", factor=4.0), dict(scaling="base", factor=8.0),
            dict(scaling="parts", factor=16.0, original=4096.0),
            dict(scaling="parts", factor=8.0, original=8192.0, fast=4.0, slow=0.0, base=500000.0)]


@pytest.mark.parametrize("args", SCALINGS)
@pytest.mark.parametrize("n", [16, 64, 128, 512])
def test_rope_table(dhs, n, args):
    """The table against the formulas; a pair's angle at far positions."""
    got = dhs.rope_table(n, **args)
    f = frequencies(n, **args)
    turns = torch.from_numpy(got).double() * 2.0 ** -64
    turns = torch.where(turns < 0, turns + 1, turns)
    want = f / (2 * math.pi)
    assert bool(((turns - want).abs() <= 2.0 ** -49 * want + 2.0 ** -64).all())


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("pairs", ["half", "interleaved"])
@pytest.mark.parametrize("shape", [(1, 1, 16, 0, 16), (3, 16, 576, 512, 64), (130, 5, 128, 0, 128),
                                   (700, 3, 96, 8, 64), (2, 128, 80, 64, 16), (1, 3, 4096, 0, 4096),
                                   (5, 2, 200, 24, 112)])
@pytest.mark.parametrize("in_place", [False, True])
def test_rotate(dhs, shape, pairs, dtype, in_place):
    n, heads, elems, offset, rotary = shape
    g = torch.Generator("cuda").manual_seed(n)
    x = torch.randn(n, heads, elems, generator=g, device="cuda").to(TYPES[dtype])
    at = torch.randint(0, 1 << 20, (n,), generator=g, device="cuda", dtype=torch.int32)
    at[0] = 0
    table = torch.from_numpy(dhs.rope_table(rotary)).cuda()
    pool = pool_of(dhs)
    before = x.clone()
    out = x if in_place else torch.full_like(x, 7.0)
    st = dhs.make_rotate(x, at, table, out=out, offset=offset, rotary=rotary, pairs=pairs, amplitude=1.25)
    assert pool.rotate(st) == 0
    torch.cuda.synchronize()
    end = offset + rotary
    want, m = turned(before[..., offset:end], at, frequencies(rotary), pairs, 1.25)
    err = (out[..., offset:end].double() - want).abs()
    assert bool((err <= 2.0 ** -21 * m * 1.25 + 1.01 * U[dtype] * want.abs() + 2.0 ** -25).all())
    assert torch.equal(out[..., :offset], before[..., :offset])
    assert torch.equal(out[..., end:], before[..., end:])
    if not in_place:
        assert torch.equal(x, before)


@pytest.mark.parametrize("pairs", ["half", "interleaved"])
def test_rotate_far_and_negative_positions(dhs, pairs):
    """Positions up to 2^31 - 1 and down to -2^31: in 64 bits a double's own
    product is off by 2^-22 there, which the bound allows for."""
    at = torch.tensor([0, 1, -1, 123456789, 2 ** 31 - 1, -2 ** 31, 1 << 24, (1 << 24) + 1],
                      dtype=torch.int64, device="cuda").to(torch.int32)
    x = torch.randn(8, 4, 64, device="cuda", generator=torch.Generator("cuda").manual_seed(3)).half()
    out = torch.empty_like(x)
    table = torch.from_numpy(dhs.rope_table(64)).cuda()
    assert pool_of(dhs).rotate(dhs.make_rotate(x, at, table, out=out, pairs=pairs)) == 0
    torch.cuda.synchronize()
    want, m = turned(x, at, frequencies(64), pairs)
    assert bool(((out.double() - want).abs() <= 2.0 ** -18 * m + 1.01 * U["f16"] * want.abs() + 2.0 ** -25).all())


@pytest.mark.parametrize("pairs", ["half", "interleaved"])
def test_rotate_inverse_is_its_gradient(dhs, pairs):
    """The inverse against the transpose (the formula's gradient) and against
    differences of the rotation along random directions."""
    g = torch.Generator("cuda").manual_seed(5)
    x = torch.randn(40, 3, 128, generator=g, device="cuda").half()
    d = torch.randn(40, 3, 128, generator=g, device="cuda").half()
    at = torch.randint(0, 100000, (40,), generator=g, device="cuda", dtype=torch.int32)
    table = torch.from_numpy(dhs.rope_table(64)).cuda()
    pool = pool_of(dhs)

    def rotate(t, inverse=False):
        y = torch.empty_like(t)
        st = dhs.make_rotate(t, at, table, out=y, offset=32, rotary=64, pairs=pairs, inverse=inverse,
                             amplitude=1.5)
        assert pool.rotate(st) == 0
        torch.cuda.synchronize()
        return y

    grad = rotate(d, inverse=True)
    want, m = turned(d[..., 32:96], at, frequencies(64), pairs, 1.5, inverse=True)
    assert bool(((grad[..., 32:96].double() - want).abs() <=
                 2.0 ** -20 * m + 1.01 * U["f16"] * want.abs() + 2.0 ** -25).all())
    # <R x, d> = <x, R^T d>, by differences R(x + h) - R(x) = R(h) too
    y = rotate(x).double()
    lhs, rhs = (y * d.double()).sum((1, 2)), (x.double() * grad.double()).sum((1, 2))
    size = y.norm(dim=(1, 2)) * d.double().norm(dim=(1, 2)) + x.double().norm(dim=(1, 2)) * grad.double().norm(dim=(1, 2))
    assert bool(((lhs - rhs).abs() <= 1.1 * U["f16"] * size).all())
    h = torch.randn(40, 3, 128, generator=g, device="cuda").half()
    step = (rotate((x.float() + h.float()).half()).double() - y) * d.double()
    by_gradient = ((x.float() + h.float()).half().double() - x.double()) * grad.double()
    assert bool(((step.sum((1, 2)) - by_gradient.sum((1, 2))).abs() <= 4 * U["f16"] * (size + 1) * 3).all())


def test_rotate_strides(dhs):
    """Head-major and misaligned slices; nothing beside them is written; a head
    stride of zero on the way in."""
    g = torch.Generator("cuda").manual_seed(6)
    table = torch.from_numpy(dhs.rope_table(32)).cuda()
    at = torch.arange(9, dtype=torch.int32, device="cuda") * 1000
    pool = pool_of(dhs)
    for off in (0, 1, 8):
        xb = torch.randn(9 * 4 * 90 + 16, generator=g, device="cuda").bfloat16()
        yb = torch.full((9 * 4 * 70 + 16,), 3.0, device="cuda").bfloat16()
        x = torch.as_strided(xb, (9, 4, 64), (90, 9 * 90, 1), off)
        y = torch.as_strided(yb, (9, 4, 64), (70, 9 * 70, 1), off)
        for src in (x, x[:, :1].expand(9, 4, 64)):
            st = dhs.make_rotate(src, at, table, out=y, offset=16, rotary=32)
            assert pool.rotate(st) == 0
            torch.cuda.synchronize()
            want, m = turned(src[..., 16:48], at, frequencies(32), "half")
            err = (y[..., 16:48].double() - want).abs()
            assert bool((err <= 2.0 ** -21 * m + 1.01 * U["bf16"] * want.abs() + 2.0 ** -25).all())
            assert torch.equal(y[..., :16], src[..., :16]) and torch.equal(y[..., 48:], src[..., 48:])
        y.fill_(3.0)
        assert bool((yb == 3.0).all())


def test_rotate_on_another_stream_and_captured(dhs):
    side = torch.cuda.Stream()
    pool = pool_of(dhs)
    table = torch.from_numpy(dhs.rope_table(64)).cuda()
    x = torch.randn(20, 2, 64, device="cuda").bfloat16()
    at = torch.arange(20, dtype=torch.int32, device="cuda")
    out = torch.zeros_like(x)
    st = dhs.make_rotate(x, at, table, out=out)
    torch.cuda.synchronize()
    assert pool.rotate_on(st, side.cuda_stream) == 0
    torch.cuda.synchronize()
    first = out.clone()
    assert pool.rotate_on(st, None) == dhs.DHS_EINVAL
    with torch.cuda.stream(side):
        graph = torch.cuda.CUDAGraph()
        graph.capture_begin()
        assert pool.rotate_on(st, side.cuda_stream) == 0
        graph.capture_end()
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, first)
        x.mul_(2)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, first * 2)


# ------------------------------------------------------------------ packing

def inputs(lay, n, seed, size=1.0):
    g = torch.Generator("cuda").manual_seed(seed)
    t = lambda m: (torch.randn(n, lay.kv, m, generator=g, device="cuda") * size *  # noqa: E731
                   torch.exp2(torch.randint(-6, 7, (n, lay.kv, 1), generator=g, device="cuda").float())).to(lay.type)
    return t(lay.key8), t(lay.wide) if lay.wide else None, None if lay.shared else t(lay.value)


def pack(dhs, pool, lay, key, wide, value, n, **kw):
    rows = torch.full((n, lay.row_bytes), 0xA5, dtype=torch.uint8, device="cuda")
    item = dhs.pack_item(n, key, wide=wide, value=value, positions=kw.pop("positions", None), rows=rows)
    st, keep = dhs.make_pack([item], lay.rows(dhs), **kw)
    assert pool.pack(st) == 0
    torch.cuda.synchronize()
    return rows


def expected(lay, key, wide, value):
    """The rows' bytes by the rule, from elements in 64 bits."""
    kc, ks = codes_of(key.double())
    scales, vc = [ks], None
    if not lay.shared:
        vc, vs = codes_of(value.double())
        scales.append(vs)
    return lay.assemble(kc, vc, wide, torch.cat(scales, 1))


@pytest.mark.parametrize("n", [1, 3, 130])
@pytest.mark.parametrize("name", sorted(LAYOUTS))
def test_pack_is_the_rule_to_the_bit(dhs, name, n):
    lay = LAYOUTS[name]
    key, wide, value = inputs(lay, n, n)
    got = pack(dhs, pool_of(dhs), lay, key, wide, value, n)
    assert torch.equal(got, expected(lay, key, wide, value))


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_pack_edges(dhs, dtype):
    """Zeros of both signs, ties, largest elements at and beside 448 2^e, tiny
    and huge ones, infinities and NaN."""
    lay = Layout(1, 16, 16, dtype=dtype)
    big = 2.0 ** 15 if dtype == "f16" else 2.0 ** 127
    small = 2.0 ** -24 if dtype == "f16" else 2.0 ** -133
    lines = [[0.0] * 16, [-0.0] * 16, [448.0, 17.0, 18.0, 19.0, 1.0625, 1.1875, -1.0625, 2.0 ** -9, 2.0 ** -10,
                                       3 * 2.0 ** -11, -2.0 ** -10, 0.0, -0.0, 464.0 / 2, 240.0, 208.0],
             [450.0] + [1.0] * 15, [449.0 * 2 ** -5] + [-1.0] * 15, [big] * 16, [small] * 16,
             [small * 3, -small] * 8, [math.inf, -math.inf, math.nan, 1.0] * 4, [math.nan] * 16,
             [math.inf] * 8 + [0.0] * 8, [1e-3, 65504.0] * 8]
    x = torch.tensor(lines, device="cuda", dtype=torch.float64).to(lay.type)[:, None]
    got = pack(dhs, pool_of(dhs), lay, x, None, x.flip(0), len(x))
    want = expected(lay, x, None, x.flip(0))
    nan = lambda r: (r[:, :32] & 127) == 127  # noqa: E731
    assert torch.equal(nan(got), nan(want))
    got[:, :32][nan(got)], want[:, :32][nan(want)] = 0, 0
    assert torch.equal(got, want)
    key, _ = lay.numbers(pack(dhs, pool_of(dhs), lay, x, None, x, len(x)))
    bad = ~torch.isfinite(x.double())
    assert bool(key[bad].isnan().all()) and bool(torch.isfinite(key[~bad]).all())


def test_pack_strides_and_items(dhs):
    """Head-major, misaligned inputs, items of 0 and more rows, more than one
    launch table; nothing past the rows is written."""
    lay = LAYOUTS["grouped_wide"]
    g = torch.Generator("cuda").manual_seed(4)
    pool = pool_of(dhs)
    for off in (0, 1):
        n = 70
        make = lambda m, s: torch.as_strided(  # noqa: E731
            torch.randn(lay.kv * n * s + 8, generator=g, device="cuda").to(lay.type), (n, lay.kv, m), (s, n * s, 1), off)
        key, wide, value = make(lay.key8, 150), make(lay.wide, 70), make(lay.value, 130)
        strides = dict(key_strides=(150, n * 150), wide_strides=(70, n * 70), value_strides=(130, n * 130))
        rows = pack(dhs, pool, lay, key, wide, value, n, **strides)
        assert torch.equal(rows, expected(lay, key, wide, value))
    key, wide, value = inputs(lay, 900, 9)
    out = torch.full((1000, lay.row_bytes), 0xA5, dtype=torch.uint8, device="cuda")
    items, at = [], 0
    for i in range(600):
        n = (i * 7) % 4 if at < 890 else 0
        items.append(dhs.pack_item(n, key[at:], wide=wide[at:], value=value[at:], rows=out[at:]))
        at += n
    st, keep = dhs.make_pack(items, lay.rows(dhs))
    assert pool.pack(st) == 0
    torch.cuda.synchronize()
    assert torch.equal(out[:at], expected(lay, key, wide, value)[:at])
    assert bool((out[at:] == 0xA5).all())


@pytest.mark.parametrize("pairs", ["half", "interleaved"])
@pytest.mark.parametrize("name,offset,rotary", [
    ("latent", 512, 64), ("grouped", 0, 128), ("grouped", 64, 64), ("grouped_f16", 8, 80),
    ("grouped_wide", 128, 64), ("grouped_wide", 0, 32), ("grouped_some_wide", 48, 16),
    ("no_wide", 16, 560), ("latent_f16", 544, 32), ("odd", 48, 32)])
def test_pack_turned(dhs, name, offset, rotary, pairs):
    """Rotated rows: the rule's number for the exact element, but for elements
    that the rotation's error carries over a border."""
    lay, n = LAYOUTS[name], 200
    key, wide, value = inputs(lay, n, 7)
    at = torch.randint(0, 1 << 18, (n,), device="cuda", dtype=torch.int32,
                       generator=torch.Generator("cuda").manual_seed(1))
    args = dict(scaling="parts", factor=8.0, original=4096.0)
    table = torch.from_numpy(dhs.rope_table(rotary, **args)).cuda()
    rows = pack(dhs, pool_of(dhs), lay, key, wide, value, n, positions=at, turns=table, pairs=pairs,
                rotary_offset=offset, rotary_elems=rotary, amplitude=1.1)
    every = key.double() if wide is None else torch.cat([key, wide], -1).double()
    end = offset + rotary
    exact, m = turned(every[..., offset:end], at, frequencies(rotary, **args), pairs, 1.1)
    err = torch.zeros_like(every)
    err[..., offset:end] = 2.0 ** -20 * m
    every[..., offset:end] = exact
    got, got_value = lay.numbers(rows)
    if lay.wide:
        w = slice(lay.key8, lay.key)
        assert bool(((got[..., w] - every[..., w]).abs() <=
                     err[..., w] + 1.01 * U[lay.dtype] * every[..., w].abs() + 2.0 ** -25).all())
    x, e = every[..., :lay.key8], err[..., :lay.key8]
    scale = rows[:, lay.off_scale:lay.off_scale + 4 * lay.kv].contiguous().view(torch.float32).double()[..., None]
    top = x.abs().amax(-1, keepdim=True) / scale  # 224 < top <= 448, but for the rotation's error
    slack = e.amax(-1, keepdim=True) / scale
    assert bool(((top <= 448 + slack) & (top > 224 - slack)).all())
    size = torch.exp2(torch.floor(torch.log2((x.abs() / scale + e / scale).clamp(min=2.0 ** -6))))
    assert bool(((got[..., :lay.key8] - x).abs() <= e + size / 16 * scale).all())
    if not lay.shared:
        assert torch.equal(got_value, lay.numbers(expected(lay, key, wide, value))[1])


# ------------------------------------------------------------------ reading back

def unpacked(dhs, pool, lay, items, shape, **kw):
    st, keep = dhs.make_unpack(items, lay.rows(dhs), **kw)
    rc = pool.unpack(st)
    torch.cuda.synchronize()
    return rc


def to_type(lay, x):
    return x.to(lay.type)


@pytest.mark.parametrize("n", [1, 5, 130])
@pytest.mark.parametrize("name", sorted(LAYOUTS))
def test_unpack_rows(dhs, name, n):
    lay = LAYOUTS[name]
    rows = lay.random(n, torch.Generator("cuda").manual_seed(n), -20, 9)
    rows[0, 0] = 0x7F
    k = torch.full((n, lay.kv, lay.key), 7.0, device="cuda").to(lay.type)
    v = torch.full((n, lay.kv, lay.value), 7.0, device="cuda").to(lay.type)
    assert unpacked(dhs, pool_of(dhs), lay, [dhs.unpack_item(n, k, value=v, rows=rows)], None) == 0
    key, value = lay.numbers(rows)
    assert torch.equal(k.nan_to_num(99), key.to(lay.type).nan_to_num(99))
    assert torch.equal(v.nan_to_num(99), value.to(lay.type).nan_to_num(99))
    assert bool(k[0, 0, 0].isnan())


class Arenas:
    def __init__(self, dhs, lay, R=2, T=20, B=50, pages=12):
        self.g = torch.Generator("cuda").manual_seed(2)
        self.sizes = [R * B, R * T, pages * PAGE]
        self.arenas = [lay.random(n, self.g) for n in self.sizes]
        self.pool = dhs.Pool(max_requests=R, sources=1, row_bytes=lay.row_bytes, page_rows=PAGE, tail_rows=T,
                             hot_rows=B, max_queries=8, max_topk=64, max_rows_per_request=4096,
                             optional_pages=pages, arenas=[a.view(-1) for a in self.arenas])


@pytest.mark.parametrize("name", ["latent", "grouped", "odd"])
def test_unpack_located(dhs, name):
    """Every tier, entries without a row, past a list's end and out of arena."""
    lay = LAYOUTS[name]
    env = Arenas(dhs, lay)
    hot, tail, opt = env.sizes
    n = 300
    tier = torch.randint(0, 3, (n,), generator=env.g, device="cuda")
    size = torch.tensor([tail, opt, hot], device="cuda")[tier]
    at = (torch.rand(n, generator=env.g, device="cuda") * size).long()
    loc = (tier << 30) + at
    first = torch.tensor([0, tail, tail + opt], device="cuda")
    want = torch.cat([env.arenas[1], env.arenas[2], env.arenas[0]])[first[tier] + at]
    loc[7], loc[9] = 0xFFFFFFFF, 0xFFFFFFFE
    lt = loc.to(torch.int32)
    k = torch.full((n, lay.kv, lay.key), 7.0, device="cuda").to(lay.type)
    v = torch.full((n, lay.kv, lay.value), 7.0, device="cuda").to(lay.type)
    item = dhs.unpack_item(n, k, value=v, loc=lt)
    assert unpacked(dhs, env.pool, lay, [item], None) == 0
    assert env.pool.status() == (0, 0)
    key, value = (x.to(lay.type) for x in lay.numbers(want))
    key[7], value[7], key[9], value[9] = 0, 0, 7, 7
    assert torch.equal(k, key) and torch.equal(v, value)
    lt[0], lt[n - 1] = tail, torch.tensor((2 << 30) + hot, device="cuda").to(torch.int32)
    lt[5] = torch.tensor(0xC0000000, device="cuda").to(torch.int32)
    key[0], key[5], key[n - 1], value[0], value[5], value[n - 1] = 0, 0, 0, 0, 0, 0
    assert unpacked(dhs, env.pool, lay, [item], None) == 0
    assert torch.equal(k, key) and torch.equal(v, value)
    assert env.pool.status() == (dhs.DHS_ERANGE, dhs.DHS_STATUS_ELOC)


def test_unpack_strides_and_one_output(dhs):
    """Keys alone or values alone, head-major into wider, misaligned buffers."""
    for name in ("grouped_wide", "latent"):
        lay, n = LAYOUTS[name], 37
        rows = lay.random(n, torch.Generator("cuda").manual_seed(1))
        key, value = (x.to(lay.type) for x in lay.numbers(rows))
        for off in (0, 3, 8):
            kb = torch.full((lay.kv * n * (lay.key + 10) + 8,), 3.0, device="cuda").to(lay.type)
            vb = torch.full((lay.kv * n * (lay.value + 6) + 8,), 3.0, device="cuda").to(lay.type)
            k = torch.as_strided(kb, (n, lay.kv, lay.key), (lay.key + 10, n * (lay.key + 10), 1), off)
            v = torch.as_strided(vb, (n, lay.kv, lay.value), (lay.value + 6, n * (lay.value + 6), 1), off)
            strides = dict(key_strides=k.stride()[:2], value_strides=v.stride()[:2])
            pool = pool_of(dhs)
            assert unpacked(dhs, pool, lay, [dhs.unpack_item(n, k, rows=rows)], None, **strides) == 0
            assert torch.equal(k, key) and bool((vb == 3.0).all())
            k.fill_(3.0)
            assert bool((kb == 3.0).all())
            assert unpacked(dhs, pool, lay, [dhs.unpack_item(n, None, value=v, rows=rows)], None, **strides) == 0
            assert torch.equal(v, value) and bool((kb == 3.0).all())


@pytest.mark.parametrize("window", [False, True])
@pytest.mark.parametrize("name", ["latent", "grouped_f16"])
def test_append_and_read_a_history(dhs, name, window):
    """Rows admitted packed, more appended through the ring by dhs_append_packed
    (rotated, several requests, more than a ring in all), read back by number:
    ring, pages and host rows."""
    lay, T, lens = LAYOUTS[name], 24, [0, 5, 130, 300]
    R, n = len(lens), 400
    g = torch.Generator("cuda").manual_seed(3)
    rows = torch.stack([lay.random(n, g) for _ in range(R)])
    pool = dhs.Pool(max_requests=R, sources=1, row_bytes=lay.row_bytes, page_rows=PAGE, tail_rows=T,
                    hot_rows=16, max_queries=8, max_topk=16, max_rows_per_request=n, optional_pages=40)
    host = torch.zeros(R, n * lay.row_bytes, dtype=torch.uint8).pin_memory()
    for r, x in enumerate(lens):
        if window:
            m = min(x, T)
            assert pool.admit_window(r, 0, rows[r, x - m:].data_ptr(), x) == 0
        else:
            mask = (torch.arange(x // PAGE) % 3 != 1).numpy()
            assert pool.admit_device(r, 0, rows[r].data_ptr(), host[r].data_ptr(), x, mask)[0] == 0
    table = torch.from_numpy(dhs.rope_table(16)).cuda()
    new = 0
    for count in (1, 24, 3, 17):
        key, wide, value = inputs(lay, R * count, count)
        at = torch.arange(R * count, dtype=torch.int32, device="cuda") * 91
        cut = lambda t, r: None if t is None else t[r * count:]  # noqa: E731
        args = dict(rotary_offset=lay.key - 16 if lay.wide else 0, rotary_elems=16, turns=table)
        its = [dhs.pack_item(count, cut(key, r), wide=cut(wide, r), value=cut(value, r), positions=cut(at, r),
                             req=r) for r in range(R)]
        st, keep = dhs.make_pack(its, lay.rows(dhs), **args)
        assert pool.append_packed(st) == 0
        packed = pack(dhs, pool, lay, key, wide, value, R * count, positions=at, **args)
        for r, x in enumerate(lens):
            rows[r, x + new:x + new + count] = packed[r * count:(r + 1) * count]
        new += count
    total = [x + new for x in lens]
    for lo, hi in ((0, 10 ** 9), (3, 150), (10 ** 9, 10 ** 9)):
        its, outs = [], []
        for r, L in enumerate(total):
            a = max(L - T if window else 0, min(lo, L))
            b = max(a, min(hi, L))
            k = torch.full((b - a + 1, lay.kv, lay.key), 7.0, device="cuda").to(lay.type)
            v = torch.full((b - a + 1, lay.kv, lay.value), 7.0, device="cuda").to(lay.type)
            its.append(dhs.unpack_item(b - a, k, value=v, req=r, first=a, flags=dhs.DHS_UNPACK_HISTORY))
            outs.append((r, a, b, k, v))
        assert unpacked(dhs, pool, lay, its, None) == 0
        for r, a, b, k, v in outs:
            key, value = (x.to(lay.type) for x in lay.numbers(rows[r, a:b]))
            assert torch.equal(k[:-1], key) and torch.equal(v[:-1], value), (r, a, b)
            assert bool((k[-1] == 7).all()) and bool((v[-1] == 7).all())
    if not window:  # written through: the host has every appended row
        for r, x in enumerate(lens):
            assert torch.equal(host[r].view(n, -1)[x:x + new], rows[r, x:x + new].cpu())
    assert pool.status() == (0, 0)


def test_unpack_on_another_stream(dhs):
    """Ordered after the pool's work, and before its next change of rows."""
    lay = LAYOUTS["latent"]
    main, side = torch.cuda.Stream(), torch.cuda.Stream()
    g = torch.Generator("cuda").manual_seed(3)
    rows, other = lay.random(3000, g), lay.random(24, g)
    host = torch.zeros(3100 * lay.row_bytes, dtype=torch.uint8).pin_memory()
    pool = dhs.Pool(max_requests=1, sources=1, row_bytes=lay.row_bytes, page_rows=PAGE, tail_rows=24,
                    hot_rows=16, max_queries=8, max_topk=16, max_rows_per_request=3100, optional_pages=200,
                    stream=main)
    torch.cuda.synchronize()
    assert pool.admit_device(0, 0, rows.data_ptr(), host.data_ptr(), 3000)[0] == 0
    k = torch.zeros(3000, 1, 576, dtype=torch.bfloat16, device="cuda")
    torch.cuda.synchronize()
    st, keep = dhs.make_unpack([dhs.unpack_item(3000, k, req=0, first=0, flags=dhs.DHS_UNPACK_HISTORY)],
                               lay.rows(dhs))
    assert pool.unpack_on(st, side.cuda_stream) == 0
    a = dhs.dhs_append_item()
    a.count, a.rows_dev = 24, other.data_ptr()
    assert pool.append([a]) == 0  # the ring's rows change behind the reading
    torch.cuda.synchronize()
    assert torch.equal(k, lay.numbers(rows)[0].bfloat16())
    assert pool.unpack_on(st, None) == dhs.DHS_EINVAL


# ----------------------------------------------------------------- refusals

def test_rotate_refusals(dhs):
    pool = pool_of(dhs)
    x = torch.zeros(4, 2, 64, device="cuda").bfloat16()
    y = torch.zeros(4, 2, 64, device="cuda").bfloat16()
    at = torch.zeros(4, dtype=torch.int32, device="cuda")
    table = torch.from_numpy(dhs.rope_table(64)).cuda()
    E = dhs.DHS_EINVAL
    for change in (dict(dtype=2), dict(tokens=-1), dict(heads=-1), dict(head_elems=60), dict(head_elems=0),
                   dict(rotary_elems=0), dict(rotary_elems=8), dict(rotary_elems=72), dict(rotary_offset=8),
                   dict(rotary_offset=-8), dict(rotary_offset=4), dict(pairs=2), dict(flags=2),
                   dict(amplitude=math.inf), dict(x_dev=None), dict(y_dev=None), dict(position_dev=None),
                   dict(turns_dev=None), dict(turns_dev=table.data_ptr() + 4), dict(x_dev=x.data_ptr() + 1),
                   dict(position_dev=at.data_ptr() + 2), dict(x_token_stride=1 << 50),
                   dict(y_dev=x.data_ptr(), y_token_stride=64)):
        st = dhs.make_rotate(x, at, table, out=y)
        for k, v in change.items():
            setattr(st, k, v)
        assert pool.rotate(st) == E, change
    st = dhs.make_rotate(x, at, table, out=y)
    st.tokens = 0
    st.x_dev = st.y_dev = st.position_dev = None
    assert pool.rotate(st) == 0
    with pytest.raises(ValueError):
        dhs.make_rotate(x.float(), at, table)
    with pytest.raises(ValueError):
        dhs.make_rotate(x, at.long(), table)
    with pytest.raises(ValueError):
        dhs.make_rotate(x, at[:3], table)
    with pytest.raises(ValueError):
        dhs.make_rotate(x, at, table[:8])
    with pytest.raises(ValueError):
        dhs.make_rotate(x.transpose(1, 2), at, table)


def test_pack_and_unpack_refusals(dhs):
    lay = LAYOUTS["grouped_wide"]
    key, wide, value = inputs(lay, 4, 1)
    at = torch.zeros(4, dtype=torch.int32, device="cuda")
    table = torch.from_numpy(dhs.rope_table(64)).cuda()
    rows = torch.zeros(4, lay.row_bytes, dtype=torch.uint8, device="cuda")
    host = torch.zeros(64 * lay.row_bytes, dtype=torch.uint8).pin_memory()
    pool = pool_of(dhs, lay.row_bytes, max_requests=2)
    other = pool_of(dhs, lay.row_bytes + 16)
    assert pool.admit_device(0, 0, rows.data_ptr(), host.data_ptr(), 4)[0] == 0
    E, S = dhs.DHS_EINVAL, dhs.DHS_ESTATE

    def attempt(how, item=(), step=(), layout=(), p=pool, n_items=1, **kw):
        it = dhs.pack_item(4, key, wide=wide, value=value, positions=at, rows=rows)
        for k, v in dict(item).items():
            setattr(it, k, v)
        st, keep = dhs.make_pack([it] * n_items, lay.rows(dhs),
                                 **{**dict(rotary_offset=128, rotary_elems=64, turns=table), **kw})
        for k, v in dict(step).items():
            setattr(st, k, v)
        for k, v in dict(layout).items():
            setattr(st.rows, k, v)
        return getattr(p, how)(st)

    for how in ("pack", "append_packed"):
        assert attempt(how) == 0
        for change in (dict(count=-1), dict(key_dev=None), dict(wide_dev=None), dict(value_dev=None),
                       dict(position_dev=None), dict(key_dev=key.data_ptr() + 1),
                       dict(position_dev=at.data_ptr() + 2)):
            assert attempt(how, change) == E, (how, change)
        for change in (dict(rotary_elems=8), dict(rotary_elems=-16), dict(rotary_offset=120),
                       dict(rotary_offset=96), dict(rotary_offset=-64), dict(pairs=3), dict(n_items=-1),
                       dict(amplitude=math.nan), dict(turns_dev=None), dict(key_token_stride=-(1 << 45))):
            assert attempt(how, step=change) == E, (how, change)
        for change in (dict(dtype=7), dict(kv_heads=0), dict(key_elems=584), dict(wide_elems=4),
                       dict(value_elems=8), dict(shared=-1), dict(kv_heads=70000)):
            assert attempt(how, layout=change) == E, (how, change)
    for change in (dict(rows_dev=None), dict(rows_dev=rows.data_ptr() + 8)):
        assert attempt("pack", change) == E
    assert attempt("pack", p=other) == 0 and attempt("append_packed", p=other) == E
    assert attempt("append_packed", dict(req=1)) == S and attempt("append_packed", dict(req=2)) == E
    assert attempt("append_packed", dict(count=9)) == E  # more than the ring
    assert attempt("append_packed", n_items=2) == E      # the same source twice
    assert pool.read_state(0, 0)[3][1] == 8              # refused calls appended nothing
    for _ in range(14):
        assert attempt("append_packed") == 0
    assert attempt("append_packed") == E                 # 64 rows at most

    out = torch.zeros(64, lay.kv, lay.key, device="cuda").to(lay.type)
    loc = torch.zeros(4, dtype=torch.int32, device="cuda")

    def read(p=pool, **kw):
        it = dhs.unpack_item(4, out, req=0, first=60, flags=dhs.DHS_UNPACK_HISTORY)
        for k, v in kw.items():
            setattr(it, k, v)
        st, keep = dhs.make_unpack([it], lay.rows(dhs))
        return p.unpack(st)

    assert read() == 0
    for change in (dict(first=61), dict(first=-1), dict(count=-1), dict(first=65, count=0), dict(flags=2),
                   dict(req=2), dict(src=1), dict(key_dev=out.data_ptr() + 1), dict(first=2 ** 62, count=2 ** 31 - 1),
                   dict(flags=0), dict(flags=0, rows_dev=rows.data_ptr() + 4),
                   dict(flags=0, loc_dev=loc.data_ptr() + 2)):
        assert read(**change) == E, change
    assert read(req=1) == S
    assert read(flags=0, loc_dev=loc.data_ptr()) == 0
    assert read(flags=0, rows_dev=rows.data_ptr()) == 0 and read(other, flags=0, rows_dev=rows.data_ptr()) == 0
    assert read(other, flags=0, loc_dev=loc.data_ptr()) == E
    assert read(count=0, key_dev=None) == 0
    torch.cuda.synchronize()
