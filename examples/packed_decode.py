"""Decoding with the pool's rows held in 8 bits.

A row is a token's latent part (512 elements, e4m3 codes under one scale) and its
rotary key part (64 elements in 16 bits): 656 bytes instead of 1152.  Prompts
arrive unrotated and unquantised: their rows are turned to their positions and
packed in one pass and admitted.  The first new token attends to the whole
history.  Request 0 is then forked into a second branch; every step packs and
appends a row to each request, turns the new queries in place, resolves the rows
that they select and attends to them in 8 bits where they lie.  What selects
reads the new rows back in 16 bits.  Half-way request 1 finishes: its pages are
released and the pool is compacted.

    python examples/packed_decode.py [--steps 8] [--rows 6000] [--check]

--check compares every output with the same attention in float64 on the CPU over
the rows as they were read back ("error"), and these with the rows that came,
turned in float64 ("held").
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from hierarchical_sparse_kv_dhs_gb300 import dhs  # noqa: E402

CODED, ROTARY, HEADS, QUERIES, TOPK = 512, 64, 16, 2, 512
KEY, VALUE, BASE = CODED + ROTARY, CODED, 10000.0
SCALE = KEY ** -0.5


class Serving:
    """A one-source pool of packed latent rows."""

    def __init__(self, requests, rows, steps, seed=0):
        self.g = torch.Generator("cuda").manual_seed(seed)
        self.max_rows = rows + steps
        self.layout = dhs.packed_rows(key_elems=KEY, wide_elems=ROTARY, value_elems=VALUE, shared=True)
        self.bytes = dhs.dhs_packed_bytes(self.layout)
        self.pool = dhs.Pool(max_requests=requests, sources=1, row_bytes=self.bytes, page_rows=64,
                             tail_rows=128, hot_rows=2048, max_queries=QUERIES, max_topk=TOPK,
                             max_rows_per_request=self.max_rows, optional_pages=3 * rows // 64)
        self.turns = torch.from_numpy(dhs.rope_table(ROTARY, base=BASE)).cuda()
        self.host = torch.zeros(requests, self.max_rows, self.bytes, dtype=torch.uint8).pin_memory()
        self.rows, self.exact, self.len = {}, {}, {}
        self.step, self.error, self.held = 0, 0.0, 0.0
        self.work = torch.empty(0, dtype=torch.uint8, device="cuda")

    def randn(self, *shape):
        return torch.randn(*shape, generator=self.g, device="cuda").to(torch.bfloat16)

    def pack(self, items):
        return dhs.make_pack(items, self.layout, rotary_offset=CODED, rotary_elems=ROTARY,
                             pairs="interleaved", turns=self.turns)

    def arrive(self, r, first, n):
        """n new rows' latent and rotary parts, and their positions."""
        part, rope = self.randn(n, CODED), self.randn(n, ROTARY)
        at = torch.arange(first, first + n, dtype=torch.int32, device="cuda")
        self.exact[r][first:first + n, :CODED] = part
        self.exact[r][first:first + n, CODED:] = rope
        return dict(key=part, wide=rope, positions=at)

    def admit(self, r, n):
        """A prompt of n rows; half of its pages stay on the GPU."""
        self.rows[r] = torch.zeros(self.max_rows, KEY, dtype=torch.bfloat16, device="cuda")
        self.exact[r], self.len[r] = torch.zeros_like(self.rows[r]), n
        new = self.arrive(r, 0, n)
        packed = torch.empty(n, self.bytes, dtype=torch.uint8, device="cuda")
        st, _keep = self.pack([dhs.pack_item(n, rows=packed, **new)])
        dhs.check(self.pool.pack(st), "pack")
        mask = torch.rand(n // 64, generator=self.g, device="cuda") < 0.5
        rc, _ = self.pool.admit_device(r, 0, packed.data_ptr(), self.host[r].data_ptr(), n,
                                       mask.cpu().numpy())
        dhs.check(rc, "admit")
        self.read_back({r: (0, n)})

    def read_back(self, spans):
        """Rows [first, first + n) of each request in 16 bits, for what selects."""
        items = [dhs.unpack_item(n, self.rows[r][first:], req=r, first=first,
                                 flags=dhs.DHS_UNPACK_HISTORY) for r, (first, n) in spans.items()]
        st, _keep = dhs.make_unpack(items, self.layout)
        dhs.check(self.pool.unpack(st), "unpack")

    def fork(self, r, child):
        rc, _ = self.pool.fork(r, child, [self.host[child].data_ptr()])
        dhs.check(rc, "fork")
        self.rows[child], self.exact[child] = self.rows[r].clone(), self.exact[r].clone()
        self.len[child] = self.len[r]

    def finish(self, r):
        dhs.check(self.pool.release(r), "release")
        del self.rows[r], self.exact[r], self.len[r]
        rc, moved = self.pool.compact(self.pool.used())
        dhs.check(rc, "compact")
        return moved

    def append(self):
        """A new row of each request, turned, packed and appended in one launch."""
        new = {r: self.arrive(r, n, 1) for r, n in self.len.items()}
        st, _keep = self.pack([dhs.pack_item(1, req=r, **x) for r, x in new.items()])
        dhs.check(self.pool.append_packed(st), "append")
        self.read_back({r: (n, 1) for r, n in self.len.items()})
        for r in self.len:
            self.len[r] += 1

    def queries(self, n):
        """n new queries of every request, their rotary parts turned to its last positions."""
        q = {r: self.randn(n, HEADS, KEY) for r in self.rows}
        for r, x in q.items():
            at = torch.arange(self.len[r] - n, self.len[r], dtype=torch.int32, device="cuda")
            st = dhs.make_rotate(x, at, self.turns, offset=CODED, rotary=ROTARY, pairs="interleaved")
            dhs.check(self.pool.rotate(st), "rotate")
        return q

    def attend(self, items):
        st, _keep = dhs.make_attend_packed(items, self.layout, heads=HEADS, scale=SCALE)
        need = self.pool.attend_packed_bytes(st)
        if self.work.numel() < need:
            self.work = torch.empty(need, dtype=torch.uint8, device="cuda")
        st.work_dev, st.work_bytes = self.work.data_ptr(), self.work.numel()
        dhs.check(self.pool.attend_packed(st), "attend")

    def dense(self, check):
        """One new token of each request over its whole history."""
        q = self.queries(1)
        out = {r: torch.empty(1, HEADS, VALUE, dtype=torch.bfloat16, device="cuda") for r in q}
        self.attend([dhs.attend_item(req=r, queries=1, q=q[r], out=out[r],
                                     flags=dhs.DHS_ATTEND_HISTORY) for r in q])
        for r in q if check else ():
            self.compare(q[r][0], self.rows[r][:self.len[r]], out[r][0])

    def sparse(self, check):
        """A step of every request: append, resolve the selected rows, attend to them."""
        self.append()
        self.step += 1
        finds, reads, got = [], [], {}
        for r, q in self.queries(QUERIES).items():
            score = q.float().mean(1) @ self.rows[r][:self.len[r]].float().T
            sel = score.topk(TOPK).indices.int()
            loc = torch.empty(QUERIES, TOPK, dtype=torch.int32, device="cuda")
            cnt = torch.empty(8, dtype=torch.int32, device="cuda")
            out = torch.empty(QUERIES, HEADS, VALUE, dtype=torch.bfloat16, device="cuda")
            it = dhs.dhs_item()
            it.req, it.queries, it.topk = r, QUERIES, TOPK
            it.sel_dev, it.loc_dev, it.counters_dev = sel.data_ptr(), loc.data_ptr(), cnt.data_ptr()
            finds.append(it)
            reads.append(dhs.attend_item(req=r, queries=QUERIES, topk=TOPK, q=q, out=out, loc=loc))
            got[r] = (q, sel, loc, cnt, out)
        st, _keep = dhs.make_step(self.step, finds)
        dhs.check(self.pool.resolve(st), "resolve")
        self.attend(reads)
        for r, (q, sel, _loc, _cnt, out) in got.items() if check else ():
            for i in range(QUERIES):
                self.compare(q[i], self.rows[r][sel[i].long()], out[i])

    def compare(self, q, rows, out):
        x = rows.double().cpu()
        want = torch.softmax(SCALE * q.double().cpu() @ x.T, -1) @ x[:, :VALUE]
        err = (out.double().cpu() - want).norm() / want.norm()
        self.error = max(self.error, float(err))

    def compare_rows(self):
        """Every row that is left against the one that came."""
        f = BASE ** (-torch.arange(0, ROTARY, 2, dtype=torch.float64) / ROTARY)
        for r, n in self.len.items():
            angle = torch.arange(n, dtype=torch.float64)[:, None] * f
            want = self.exact[r][:n].double().cpu()
            a, b = want[:, CODED::2].clone(), want[:, CODED + 1::2].clone()
            want[:, CODED::2] = a * angle.cos() - b * angle.sin()
            want[:, CODED + 1::2] = b * angle.cos() + a * angle.sin()
            self.rows[r].zero_()
            self.read_back({r: (0, n)})
            err = (self.rows[r][:n].double().cpu() - want).norm(dim=1) / want.norm(dim=1)
            self.held = max(self.held, float(err.max()))


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--steps", type=int, default=8)
    ap.add_argument("--rows", type=int, default=6000)
    ap.add_argument("--check", action="store_true")
    a = ap.parse_args(argv)
    if a.rows < TOPK:
        ap.error("--rows: at least %d" % TOPK)
    s = Serving(requests=3, rows=a.rows, steps=max(0, a.steps))
    s.admit(1, max(TOPK, a.rows // 2))
    s.admit(0, a.rows)
    s.dense(a.check)
    s.fork(0, 2)
    moved = 0
    for i in range(a.steps):
        if i == a.steps // 2:
            moved = s.finish(1)
        s.sparse(a.check)
    if a.check:
        s.compare_rows()
    dhs.check(s.pool.status()[0], "status")
    done = dict(steps=a.steps, requests=len(s.rows), pages=s.pool.used(), moved=moved,
                capacity=s.pool.capacity(), error=s.error if a.check else None,
                held=s.held if a.check else None)
    print("  ".join("%s %s" % kv for kv in done.items()))
    s.pool.close()
    return done


if __name__ == "__main__":
    main()
