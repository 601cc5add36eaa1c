"""Rotary positions and packed rows without a GPU: tables, sizes and refusals
on the host; the ctypes structures; the plain rule's own codes."""
import ctypes
import math

import pytest

torch = pytest.importorskip("torch")

from packed_layouts import LAYOUTS, codes_of, exponent  # noqa: E402


@pytest.fixture(scope="module")
def dhs():
    from hierarchical_sparse_kv_dhs_gb300.build import build
    build()
    from hierarchical_sparse_kv_dhs_gb300 import dhs as mod
    return mod


def test_null_arguments(dhs):
    E = dhs.DHS_EINVAL
    size, n32 = ctypes.c_size_t(0), ctypes.c_int32(7)
    rows = LAYOUTS["latent"].rows(dhs)
    pack, _ = dhs.make_pack([], rows)
    unpack, _ = dhs.make_unpack([], rows)
    attend, _ = dhs.make_attend_packed([], rows, heads=16, scale=1.0)
    rotate = dhs.dhs_rotate_step()
    for name, st in (("dhs_rotate", rotate), ("dhs_pack", pack), ("dhs_append_packed", pack),
                     ("dhs_unpack", unpack), ("dhs_attend_packed", attend)):
        assert getattr(dhs.lib, name)(None, ctypes.byref(st)) == E, name
        assert getattr(dhs.lib, name)(None, None) == E, name
    for name, st in (("dhs_rotate_on", rotate), ("dhs_unpack_on", unpack), ("dhs_attend_packed_on", attend)):
        assert getattr(dhs.lib, name)(None, ctypes.byref(st), 1) == E, name
        assert getattr(dhs.lib, name)(None, None, None) == E, name
    assert dhs.lib.dhs_attend_packed_bytes(None, ctypes.byref(attend), ctypes.byref(size)) == E
    assert dhs.lib.dhs_attend_packed_bytes(None, ctypes.byref(attend), None) == E
    assert dhs.lib.dhs_packed_bytes(None, ctypes.byref(n32)) == E and n32.value == 0
    assert dhs.lib.dhs_packed_bytes(ctypes.byref(rows), None) == E
    assert dhs.lib.dhs_rope_table(None, None) == E


def test_descriptors_match_the_header(dhs):
    """The ctypes structures have the C ones' sizes (LP64: no hidden padding)."""
    size = ctypes.sizeof
    assert size(dhs.dhs_rope_config) == 2 * 4 + 5 * 8
    assert size(dhs.dhs_rotate_step) == 10 * 4 + 4 * 8 + 4 * 8
    assert size(dhs.dhs_packed_rows) == 6 * 4
    assert size(dhs.dhs_pack_item) == 4 * 4 + 5 * 8
    assert size(dhs.dhs_pack_step) == 6 * 4 + 6 * 4 + 6 * 8 + 2 * 8
    assert size(dhs.dhs_unpack_item) == 4 * 4 + 5 * 8
    assert size(dhs.dhs_unpack_step) == 6 * 4 + 2 * 4 + 5 * 8
    assert size(dhs.dhs_attend_packed_step) == 6 * 4 + 4 * 4 + 4 * 8 + 3 * 8


@pytest.mark.parametrize("name", sorted(LAYOUTS))
def test_packed_bytes(dhs, name):
    lay = LAYOUTS[name]
    assert dhs.dhs_packed_bytes(lay.rows(dhs)) == lay.row_bytes
    assert lay.row_bytes % 16 == 0


@pytest.mark.parametrize("change", [
    dict(dtype=2), dict(kv_heads=0), dict(kv_heads=-1), dict(kv_heads=60), dict(key_elems=592),
    dict(key_elems=72), dict(key_elems=0), dict(wide_elems=4), dict(wide_elems=-8), dict(wide_elems=72),
    dict(wide_elems=576), dict(value_elems=0), dict(value_elems=520), dict(value_elems=8),
    dict(shared=1, value_elems=512, wide_elems=72), dict(shared=1, key_elems=128, wide_elems=0, value_elems=144),
    dict(shared=2)])
def test_layouts_that_are_refused(dhs, change):
    rows = dhs.packed_rows(key_elems=576, wide_elems=64, value_elems=512, kv_heads=1)
    assert dhs.dhs_packed_bytes(rows) == 512 + 512 + 128 + 16
    for k, v in change.items():
        setattr(rows, k, v)
    n = ctypes.c_int32(7)
    assert dhs.lib.dhs_packed_bytes(ctypes.byref(rows), ctypes.byref(n)) == dhs.DHS_EINVAL


def test_rope_table(dhs):
    """Each scaling against its formula, and what is refused."""
    n = 64
    f = [10000.0 ** (-2 * i / n) for i in range(n // 2)]
    stretched = [(10000.0 * 4 ** (n / (n - 2))) ** (-2 * i / n) for i in range(n // 2)]
    keep = [min(1, max(0, (2048 * x / (2 * math.pi) - 1) / 31)) for x in f]
    wants = {"plain": f, "linear": [x / 4 for x in f], "base": stretched,
             "parts": [x * k + x / 4 * (1 - k) for x, k in zip(f, keep)]}
    for scaling, want in wants.items():
        got = dhs.rope_table(n, scaling=scaling, factor=4.0, original=2048.0)
        for g, w in zip(got.tolist(), want):
            turns = (g % 2 ** 64) / 2 ** 64
            assert abs(turns - w / (2 * math.pi)) <= 2.0 ** -49 * w
    assert min(keep) == 0 and max(keep) == 1
    for kw in (dict(rotary=0), dict(rotary=8), dict(rotary=40), dict(rotary=-16), dict(base=1.0),
               dict(base=math.nan), dict(base=math.inf), dict(scaling="linear", factor=0.5),
               dict(scaling="base", factor=math.inf), dict(scaling="parts", factor=2.0),
               dict(scaling="parts", factor=2.0, original=100.0, fast=1.0, slow=1.0),
               dict(scaling="parts", factor=2.0, original=100.0, slow=-1.0),
               dict(scaling="parts", factor=math.nan, original=100.0)):
        with pytest.raises(dhs.DhsError):
            dhs.rope_table(**{**dict(rotary=64), **kw})


def test_the_rule_of_codes():
    """codes_of against the type's own cast where both round the same way."""
    g = torch.Generator().manual_seed(0)
    x = torch.randn(50, 64, generator=g, dtype=torch.float64) * \
        torch.exp2(torch.randint(-20, 20, (50, 1), generator=g).double())
    code, scale = codes_of(x)
    assert torch.equal(code, (x / scale[:, None]).float().to(torch.float8_e4m3fn).view(torch.uint8))
    top = x.abs().amax(1) / scale
    assert bool(((top <= 448) & (top > 224)).all())
    assert [exponent(t) for t in (0.0, 448.0, 448.1, 449 * 2.0 ** -3, 1.0, 1e-30, 2.0 ** 127.9)] == \
        [-64, 0, 1, -2, -8, -64, 120]
    odd = torch.tensor([[math.inf, -math.inf, math.nan, 448.0]], dtype=torch.float64)
    code, scale = codes_of(odd)
    assert code.tolist() == [[127, 127, 127, 126]] and scale.tolist() == [1.0]
