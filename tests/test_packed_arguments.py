"""What make_rotate, make_pack and make_unpack refuse before any launch: tensors
of another type, with fewer elements than the call takes, or out of the GPU's
reach.  Without a GPU: tensors on the CPU, and stand-ins for those on GPUs."""
import pytest

torch = pytest.importorskip("torch")

from packed_layouts import LAYOUTS  # noqa: E402


@pytest.fixture(scope="module")
def dhs():
    from hierarchical_sparse_kv_dhs_gb300.build import build
    build()
    from hierarchical_sparse_kv_dhs_gb300 import dhs as mod
    return mod


class OnGpu:
    """A tensor as the binding sees one, on GPU `index`."""

    def __init__(self, t, index=0):
        self.t, self.index = t, index

    is_cuda = True

    def __getattr__(self, name):
        return getattr(self.t, name)

    def get_device(self):
        return self.index


def on(t, index=0):
    return OnGpu(t, index)


LAY = LAYOUTS["grouped_wide"]  # 4 heads of 128 + 64 key and 128 value elements, bf16
N = 5


def pack_arguments():
    z = lambda m: torch.zeros(N, LAY.kv, m, dtype=torch.bfloat16)  # noqa: E731
    return dict(key=z(LAY.key8), wide=z(LAY.wide), value=z(LAY.value),
                positions=torch.zeros(N, dtype=torch.int32),
                rows=torch.zeros(N, LAY.row_bytes, dtype=torch.uint8))


def make_pack(dhs, given, turns=None, where=None, **kw):
    """A step of items of `given`, all on GPU 0 but for what `where` says."""
    put = lambda k, t: t if t is None or (where or {}).get(k) == "cpu" else on(t, (where or {}).get(k, 0))  # noqa: E731
    item = dhs.pack_item(N, **{k: put(k, t) for k, t in given.items()})
    turns = torch.zeros(32, dtype=torch.int64) if turns is None else turns
    return dhs.make_pack([item], LAY.rows(dhs), turns=put("turns", turns),
                         **{**dict(rotary_offset=128, rotary_elems=64), **kw})


def test_pack_arguments(dhs):
    good = pack_arguments()
    make_pack(dhs, good)
    make_pack(dhs, {**good, "value": good["value"].flatten()})
    make_pack(dhs, {**good, "positions": None}, rotary_elems=0)
    make_pack(dhs, {**good, "positions": good["positions"].long()}, rotary_elems=0)
    make_pack(dhs, {**good, "rows": None})
    wide = torch.zeros(N, LAY.kv, LAY.key, dtype=torch.bfloat16)
    make_pack(dhs, {**good, "key": wide, "wide": wide[..., LAY.key8:]},
              key_strides=(LAY.kv * LAY.key, LAY.key), wide_strides=(LAY.kv * LAY.key, LAY.key))
    make_pack(dhs, {**good, "key": good["key"][:1, :1]}, key_strides=(0, 0))


@pytest.mark.parametrize("name,t", [
    ("positions", torch.arange(N)), ("positions", torch.zeros(N - 1, dtype=torch.int32)),
    ("positions", torch.zeros(2 * N, dtype=torch.int32)[::2]),
    ("key", torch.zeros(N, 4, 128)), ("key", torch.zeros(N, 4, 128, dtype=torch.float16)),
    ("key", torch.zeros(N - 1, 4, 128, dtype=torch.bfloat16)),
    ("key", torch.zeros(N, 4, 192, dtype=torch.bfloat16)[..., :128]),
    ("wide", torch.zeros(N, 4, 32, dtype=torch.bfloat16)), ("wide", torch.zeros(N, 4, 64, dtype=torch.int16)),
    ("value", torch.zeros(N, 4, 64, dtype=torch.bfloat16)), ("value", torch.zeros(N, 4, 128, dtype=torch.float64)),
    ("rows", torch.zeros(N - 1, LAY.row_bytes, dtype=torch.uint8)),
    ("rows", torch.zeros(N, LAY.row_bytes + 16, dtype=torch.uint8)[:, :-16])])
def test_pack_refuses(dhs, name, t):
    with pytest.raises(ValueError, match=name):
        make_pack(dhs, {**pack_arguments(), name: t})


@pytest.mark.parametrize("turns", [torch.zeros(31, dtype=torch.int64), torch.zeros(32), torch.zeros(32, dtype=torch.float64)])
def test_pack_refuses_tables(dhs, turns):
    with pytest.raises(ValueError, match="turns"):
        make_pack(dhs, pack_arguments(), turns=turns)


@pytest.mark.parametrize("strides", [(4 * 128, 256), (4 * 128 + 1, 128), (-4 * 128, 128), (512, -128)])
def test_pack_refuses_strides_that_leave_the_tensor(dhs, strides):
    with pytest.raises(ValueError, match="key"):
        make_pack(dhs, pack_arguments(), key_strides=strides)


@pytest.mark.parametrize("where", ["cpu", 1])
@pytest.mark.parametrize("name", ["key", "wide", "value", "positions", "rows", "turns"])
def test_pack_refuses_memory_elsewhere(dhs, name, where):
    with pytest.raises(ValueError, match="GPU"):
        make_pack(dhs, pack_arguments(), where={name: where})


def unpack(dhs, flags=0, where=None, **given):
    put = lambda k, t: t if t is None or (where or {}).get(k) == "cpu" else on(t, (where or {}).get(k, 0))  # noqa: E731
    kw = given.pop("strides", {})
    item = dhs.unpack_item(N, flags=flags, **{k: put(k, t) for k, t in given.items()})
    return dhs.make_unpack([item], LAY.rows(dhs), **kw)


def unpack_arguments():
    z = lambda m: torch.zeros(N, LAY.kv, m, dtype=torch.bfloat16)  # noqa: E731
    return dict(key=z(LAY.key), value=z(LAY.value), loc=torch.zeros(N, dtype=torch.int32))


def test_unpack_arguments(dhs):
    good = unpack_arguments()
    rows = torch.zeros(N, LAY.row_bytes, dtype=torch.uint8)
    unpack(dhs, **good)
    unpack(dhs, **{**good, "key": None})
    unpack(dhs, **{**good, "loc": None}, rows=rows)
    unpack(dhs, **{**good, "loc": None}, flags=dhs.DHS_UNPACK_HISTORY)
    unpack(dhs, **{**good, "key": torch.zeros(N + 3, LAY.kv, LAY.key, dtype=torch.bfloat16)})
    unpack(dhs, **{**good, "key": torch.zeros(LAY.kv, N, LAY.key, dtype=torch.bfloat16)},
           strides=dict(key_strides=(LAY.key, N * LAY.key)))


@pytest.mark.parametrize("name,t", [
    ("loc", torch.zeros(N, dtype=torch.int64)), ("loc", torch.zeros(N - 1, dtype=torch.int32)),
    ("key", torch.zeros(N, 4, 128, dtype=torch.bfloat16)), ("key", torch.zeros(N, 4, 192, dtype=torch.float16)),
    ("value", torch.zeros(N - 1, 4, 128, dtype=torch.bfloat16)), ("value", torch.zeros(N, 4, 128)),
    ("rows", torch.zeros(N, LAY.row_bytes - 16, dtype=torch.uint8))])
def test_unpack_refuses(dhs, name, t):
    with pytest.raises(ValueError, match=name):
        unpack(dhs, **{**unpack_arguments(), name: t})


@pytest.mark.parametrize("where", ["cpu", 1])
@pytest.mark.parametrize("name", ["key", "value", "loc"])
def test_unpack_refuses_memory_elsewhere(dhs, name, where):
    with pytest.raises(ValueError, match="GPU"):
        unpack(dhs, where={name: where}, **unpack_arguments())


@pytest.mark.parametrize("where", ["cpu", 1])
@pytest.mark.parametrize("name", ["x", "out", "positions", "turns"])
def test_rotate_refuses_memory_elsewhere(dhs, name, where):
    x = torch.zeros(N, 2, 64, dtype=torch.bfloat16)
    given = dict(x=x, out=x.clone(), positions=torch.zeros(N, dtype=torch.int32),
                 turns=torch.zeros(32, dtype=torch.int64))
    assert dhs.make_rotate(**{k: on(t) for k, t in given.items()}).tokens == N
    with pytest.raises(ValueError, match="GPU"):
        dhs.make_rotate(**{k: t if k == name and where == "cpu" else on(t, where if k == name else 0)
                           for k, t in given.items()})


def test_rotate_refuses_other_tables(dhs):
    """Turns are the table's integers, not its angles."""
    x = on(torch.zeros(N, 2, 64, dtype=torch.bfloat16))
    at = on(torch.zeros(N, dtype=torch.int32))
    with pytest.raises(ValueError, match="turns"):
        dhs.make_rotate(x, at, on(torch.zeros(32, dtype=torch.float64)))
