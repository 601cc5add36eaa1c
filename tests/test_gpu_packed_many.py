"""Rotation, packing and reading back of many rows and many items at once, of
which a block has more, and of tensors whose rows lie gigabytes apart."""
import pytest
import torch

from packed_layouts import LAYOUTS
from test_gpu_packed_rows import expected, inputs, pack, pool_of, to_type
from test_gpu_packed_rows import dhs  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("name", ["grouped", "grouped_some_wide", "no_wide", "latent", "smallest"])
def test_pack_many_rows(dhs, name):  # noqa: F811
    """Enough rows that a block has all keys of its tokens."""
    lay, n = LAYOUTS[name], 21001
    key, wide, value = inputs(lay, n, 5)
    pool = pool_of(dhs)
    rows = pack(dhs, pool, lay, key, wide, value, n)
    assert torch.equal(rows, expected(lay, key, wide, value))
    # read back: codes times scales are exact in bf16, and in f16 within its range
    k = torch.zeros(n, lay.kv, lay.key, dtype=lay.type, device="cuda")
    st, keep = dhs.make_unpack([dhs.unpack_item(n, k, rows=rows)], lay.rows(dhs))
    assert pool.unpack(st) == 0
    torch.cuda.synchronize()
    assert torch.equal(k, to_type(lay, lay.numbers(rows)[0]))


@pytest.mark.parametrize("pairs", ["half", "interleaved"])
@pytest.mark.parametrize("name,offset,rotary", [("grouped", 0, 128), ("grouped_wide", 128, 64),
                                                ("no_wide", 16, 512)])
def test_pack_many_turned_rows(dhs, name, offset, rotary, pairs):  # noqa: F811
    """In one call as in calls of 100 rows: each row's bytes depend on it alone."""
    lay, n = LAYOUTS[name], 21001
    key, wide, value = inputs(lay, n, 6)
    at = torch.randint(-5, 1 << 20, (n,), device="cuda", dtype=torch.int32)
    turn = dict(rotary_offset=offset, rotary_elems=rotary, pairs=pairs,
                turns=torch.from_numpy(dhs.rope_table(rotary)).cuda())
    pool = pool_of(dhs)
    rows = pack(dhs, pool, lay, key, wide, value, n, positions=at, **turn)
    part = lambda t, i: None if t is None else t[i:i + 100]  # noqa: E731
    for i in (0, 100, 10400, 20950):
        few = pack(dhs, pool, lay, part(key, i), part(wide, i), part(value, i), min(100, n - i),
                   positions=part(at, i), **turn)
        assert torch.equal(few, rows[i:i + 100])


@pytest.mark.parametrize("name", ["latent", "grouped", "no_wide", "grouped_f16"])
def test_unpack_many_items(dhs, name):  # noqa: F811
    """More than one launch table; items of no rows; outputs that only some ask for."""
    lay = LAYOUTS[name]
    g = torch.Generator("cuda").manual_seed(2)
    rows = lay.random(2500, g)
    pool = pool_of(dhs)
    k = torch.full((2500, lay.kv, lay.key), 7.0, dtype=lay.type, device="cuda")
    v = torch.full((2500, lay.kv, lay.value), 7.0, dtype=lay.type, device="cuda")
    items, at, asked = [], 0, torch.zeros(2, 2500, dtype=torch.bool, device="cuda")
    for i in range(700):
        n = (i * 11) % 7
        items.append(dhs.unpack_item(n, k[at:] if i % 3 else None, value=v[at:] if i % 4 else None,
                                     rows=rows[at:]))
        asked[0, at:at + n], asked[1, at:at + n] = i % 3 > 0, i % 4 > 0
        at += n
    assert at < 2500
    st, keep = dhs.make_unpack(items, lay.rows(dhs))
    assert pool.unpack(st) == 0
    torch.cuda.synchronize()
    for got, want, on in zip((k, v), lay.numbers(rows), asked):
        assert torch.equal(got[on], to_type(lay, want)[on])
        assert bool((got[~on] == 7).all())


def test_rows_gigabytes_apart(dhs):  # noqa: F811
    """Offsets past 32 bits in the tensors that rows come from and go to."""
    lay, n, step = LAYOUTS["latent"], 300, 1 << 23  # elements: 16 MB from row to row
    pool = pool_of(dhs)
    far = torch.zeros(n * step, dtype=lay.type, device="cuda").as_strided((n, 1, 576), (step, 576, 1))
    near = torch.randn(n, 1, 576, device="cuda").to(lay.type)
    far.copy_(near)
    at = torch.arange(n, dtype=torch.int32, device="cuda") * 1000
    table = torch.from_numpy(dhs.rope_table(64)).cuda()
    for x in (far, near):
        assert pool.rotate(dhs.make_rotate(x, at, table, offset=512, rotary=64)) == 0
    torch.cuda.synchronize()
    assert torch.equal(far, near)
    rows = pack(dhs, pool, lay, far, far[..., 512:], None, n, key_strides=(step, 576),
                wide_strides=(step, 576))
    assert torch.equal(rows, pack(dhs, pool, lay, near, near[..., 512:], None, n,
                                  key_strides=(576, 576), wide_strides=(576, 576)))
    st, keep = dhs.make_unpack([dhs.unpack_item(n, far, rows=rows)], lay.rows(dhs),
                               key_strides=(step, 576))
    assert pool.unpack(st) == 0
    torch.cuda.synchronize()
    assert torch.equal(far, lay.numbers(rows)[0].to(lay.type))
