"""Sparse decoding of a request that branches.

Two requests are admitted to a pool.  Their first new token attends to the
whole history (a dense layer).  Request 0 is then forked into a second branch;
every step appends a row to each request, resolves the rows that its queries
select, and attends to them where they lie, without staging copies.  Half-way
request 1 finishes: its pages are released and the pool is compacted, so that
the top of the optional arena is free for other use; the branches go on.

    python examples/branch_decode.py [--steps 8] [--rows 6000] [--check]

--check compares every output with the same attention in float64 on the CPU.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from hierarchical_sparse_kv_dhs_gb300 import dhs  # noqa: E402

KEY, VALUE, HEADS, QUERIES, TOPK = 576, 512, 16, 2, 512
SCALE = KEY ** -0.5


class Serving:
    """A one-source pool of latent rows (the value is the key's beginning)."""

    def __init__(self, requests, rows, steps, seed=0):
        self.g = torch.Generator("cuda").manual_seed(seed)
        self.max_rows = rows + steps
        self.pool = dhs.Pool(max_requests=requests, sources=1, row_bytes=2 * KEY, page_rows=64,
                             tail_rows=128, hot_rows=2048, max_queries=QUERIES, max_topk=TOPK,
                             max_rows_per_request=self.max_rows, optional_pages=3 * rows // 64)
        self.host = torch.zeros(requests, self.max_rows, KEY, dtype=torch.bfloat16).pin_memory()
        self.rows, self.len, self.step, self.error = {}, {}, 0, 0.0
        self.work = torch.empty(0, dtype=torch.uint8, device="cuda")

    def randn(self, *shape):
        return torch.randn(*shape, generator=self.g, device="cuda").to(torch.bfloat16)

    def admit(self, r, n):
        """n prefilled rows; half of the pages stay on the GPU."""
        rows = self.randn(self.max_rows, KEY)
        mask = torch.rand(n // 64, generator=self.g, device="cuda") < 0.5
        rc, _ = self.pool.admit_device(r, 0, rows.data_ptr(), self.host[r].data_ptr(), n,
                                       mask.cpu().numpy())
        dhs.check(rc, "admit")
        self.rows[r], self.len[r] = rows, n

    def fork(self, r, child):
        rc, _ = self.pool.fork(r, child, [self.host[child].data_ptr()])
        dhs.check(rc, "fork")
        self.rows[child], self.len[child] = self.rows[r].clone(), self.len[r]

    def finish(self, r):
        dhs.check(self.pool.release(r), "release")
        del self.rows[r], self.len[r]
        rc, moved = self.pool.compact(self.pool.used())
        dhs.check(rc, "compact")
        return moved

    def append(self):
        items = []
        for r in self.rows:
            row = self.randn(1, KEY)
            self.rows[r][self.len[r]] = row[0]
            a = dhs.dhs_append_item()
            a.req, a.count, a.rows_dev = r, 1, self.rows[r][self.len[r]].data_ptr()
            items.append(a)
            self.len[r] += 1
        dhs.check(self.pool.append(items), "append")

    def attend(self, items):
        st, _keep = dhs.make_attend(items, heads=HEADS, key_elems=KEY, value_elems=VALUE, scale=SCALE)
        need = self.pool.attend_bytes(st)
        if self.work.numel() < need:
            self.work = torch.empty(need, dtype=torch.uint8, device="cuda")
        st.work_dev, st.work_bytes = self.work.data_ptr(), self.work.numel()
        dhs.check(self.pool.attend(st), "attend")

    def dense(self, check):
        """One new token of each request over its whole history."""
        items, got = [], {}
        for r in self.rows:
            q = self.randn(1, HEADS, KEY)
            out = torch.empty(1, HEADS, VALUE, dtype=torch.bfloat16, device="cuda")
            items.append(dhs.attend_item(req=r, queries=1, q=q, out=out,
                                         flags=dhs.DHS_ATTEND_HISTORY))
            got[r] = (q, out)
        self.attend(items)
        for r, (q, out) in got.items() if check else ():
            self.compare(q[0], self.rows[r][:self.len[r]], out[0])

    def sparse(self, check):
        """A step of every request: append, resolve the selected rows, attend to them."""
        self.append()
        self.step += 1
        finds, reads, got = [], [], {}
        for r in self.rows:
            q = self.randn(QUERIES, HEADS, KEY)
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
    dhs.check(s.pool.status()[0], "status")
    done = dict(steps=a.steps, requests=len(s.rows), pages=s.pool.used(), moved=moved,
                capacity=s.pool.capacity(), error=s.error if a.check else None)
    print("  ".join("%s %s" % kv for kv in done.items()))
    s.pool.close()
    return done


if __name__ == "__main__":
    main()
