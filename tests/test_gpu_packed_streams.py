"""Reading back and attention to packed rows, queued on another stream behind
work that keeps it busy, when the pool's own stream changes what they read; and
rotation, packing, attention and reading back as one captured step."""
import pytest
import torch

from packed_layouts import LAYOUTS
from test_gpu_packed_attend import Located, check_located, dhs  # noqa: F401
from test_gpu_packed_attend import History
from test_gpu_side_streams import busy

pytestmark = pytest.mark.gpu
N = 640


class Reads:
    """Request r read back whole, and attention to its history, into fresh outputs."""

    def __init__(self, dhs, env, r):  # noqa: F811
        self.dhs, self.env, self.r, lay = dhs, env, r, env.lay
        self.q = torch.randn(1, lay.heads, lay.key, generator=env.g, device="cuda").to(lay.type)

    def enqueue(self, stream):
        d, pool, lay = self.dhs, self.env.pool, self.env.lay
        key = torch.zeros(N, lay.kv, lay.key, dtype=lay.type, device="cuda")
        out = torch.zeros(1, lay.heads, lay.value, dtype=lay.type, device="cuda")
        rd, keep1 = d.make_unpack([d.unpack_item(N, key, req=self.r, flags=d.DHS_UNPACK_HISTORY)],
                                  lay.rows(d))
        at, keep2 = d.make_attend_packed(
            [d.attend_item(req=self.r, queries=1, q=self.q, out=out, flags=d.DHS_ATTEND_HISTORY)],
            lay.rows(d), heads=lay.heads, scale=lay.scale)
        work = torch.empty(max(256, pool.attend_packed_bytes(at)), dtype=torch.uint8, device="cuda")
        at.work_dev, at.work_bytes = work.data_ptr(), work.numel()
        torch.cuda.synchronize()  # the buffers are ready on every stream
        block = None
        if stream is None:
            assert pool.unpack(rd) == 0 and pool.attend_packed(at) == 0
        else:
            block = busy(stream)
            assert pool.unpack_on(rd, stream.cuda_stream) == 0
            assert pool.attend_packed_on(at, stream.cuda_stream) == 0
        return key, out, (work, block)


@pytest.mark.parametrize("name", ["latent", "grouped_f16"])
@pytest.mark.parametrize("change", ["admit", "append", "append_packed", "refill"])
def test_reads_on_another_stream_come_first(dhs, name, change):  # noqa: F811
    lay = LAYOUTS[name]
    env = History(dhs, lay, [N, N, N], resident=0.0 if change == "refill" else 1.0)
    pool = env.pool
    reads = Reads(dhs, env, 0)
    want = reads.enqueue(None)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    other = lay.random(N, env.g)
    new = torch.randn(24, lay.kv, lay.key, generator=env.g, device="cuda").to(lay.type)
    wide = new[..., lay.key8:].contiguous()
    value = torch.randn(24, lay.kv, lay.value, generator=env.g, device="cuda").to(lay.type)
    got = reads.enqueue(side)
    assert not side.query()  # still busy: what follows is queued behind it
    if change == "admit":  # other rows into the freed slots and the ring
        assert pool.release(0) == 0
        host = torch.zeros(N * lay.row_bytes, dtype=torch.uint8).pin_memory()
        assert pool.admit_device(0, 0, other.data_ptr(), host.data_ptr(), N, [1] * (N // 16))[0] == 0
        assert pool.flush() == 0
    elif change == "append":
        a = dhs.dhs_append_item()
        a.count, a.rows_dev = 8, other.data_ptr()
        assert pool.append([a]) == 0
    elif change == "append_packed":
        st, keep = dhs.make_pack(
            [dhs.pack_item(8, new, wide=wide if lay.wide else None, value=None if lay.shared else value)],
            lay.rows(dhs), key_strides=(lay.kv * lay.key, lay.key))
        assert pool.append_packed(st) == 0
    else:
        assert pool.refill(100)[1] > 20
        st, keep = dhs.make_attend_packed([], lay.rows(dhs), heads=lay.heads, scale=lay.scale)
        assert pool.attend_packed(st) == 0  # flushes
    torch.cuda.synchronize()
    for a, b in zip(got[:2], want[:2]):
        assert torch.equal(a.view(torch.int16), b.view(torch.int16))
    assert pool.status() == (0, 0)


def test_a_captured_step(dhs):  # noqa: F811
    """Queries turned in place, rows packed into the caller's arena, attended to and
    read back: captured once, replayed with other numbers and positions."""
    lay, n = LAYOUTS["latent"], 300
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        env = Located(dhs, lay, seed=4)
        pool, g = env.pool, env.g
        assert pool.stream == side
        turns = torch.from_numpy(dhs.rope_table(64)).cuda()
        part = torch.empty(n, 1, lay.key8, dtype=lay.type, device="cuda")
        rope = torch.empty(n, 1, lay.wide, dtype=lay.type, device="cuda")
        at = torch.empty(n, dtype=torch.int32, device="cuda")
        back = torch.empty(n, 1, lay.key, dtype=lay.type, device="cuda")
        loc = torch.arange(n, device="cuda")[None] + (1 << 30)  # the first pages' rows
        it, t = env.item(loc)
        raw = torch.empty_like(t[0])
        qat = torch.full((1,), n, dtype=torch.int32, device="cuda")
        turn = dict(offset=512, rotary=64, pairs="interleaved")
        rot = dhs.make_rotate(raw, qat, turns, out=t[0], **turn)
        apart = torch.empty_like(env.arenas[2])
        packs = [dhs.make_pack([dhs.pack_item(n, part, wide=rope, positions=at, rows=to)],
                               lay.rows(dhs), rotary_offset=512, rotary_elems=64,
                               pairs="interleaved", turns=turns)
                 for to in (env.arenas[2], apart)]
        st, keep2 = dhs.make_attend_packed([it], lay.rows(dhs), heads=lay.heads, scale=lay.scale)
        work = torch.empty(max(256, pool.attend_packed_bytes(st)), dtype=torch.uint8, device="cuda")
        st.work_dev, st.work_bytes = work.data_ptr(), work.numel()
        rd, keep3 = dhs.make_unpack([dhs.unpack_item(n, back, loc=t[3])], lay.rows(dhs))
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        graph.capture_begin()
        for rc in (pool.rotate(rot), pool.pack(packs[0][0]), pool.attend_packed(st), pool.unpack(rd)):
            assert rc == 0
        graph.capture_end()
        for seed in (1, 2):
            for x in (raw, part, rope):
                x.normal_(generator=g)
            at.copy_(torch.randint(0, 1 << 20, (n,), generator=g, device="cuda"))
            qat.fill_(seed << 19)
            for x in (t[0], t[1], t[2], back):
                x.zero_()
            graph.replay()
            turned = torch.empty_like(raw)
            assert pool.rotate(dhs.make_rotate(raw, qat, turns, out=turned, **turn)) == 0
            assert pool.pack(packs[1][0]) == 0
            check_located(env, [(loc, t)])
            assert torch.equal(t[0], turned)
            assert torch.equal(env.arenas[2][:n], apart[:n])
            assert torch.equal(back, lay.numbers(env.arenas[2][:n])[0].to(lay.type))
        assert pool.status() == (0, 0)
