"""A decode directly behind the call that wrote what it reads early.

A decode reads its page tables and the cached rows more than 32 below its new
tokens before the kernel in front of it has finished.  pkv_store,
pkv_pages_copy and pkv_tables_remap therefore let it start only once all they
wrote is visible.  Each chain below is run with a wait after every call and
then captured and replayed without one: the same bits, and the same rows in
the same pages.  What a reader too early would find (the old ids, the rows
before the copy or the store) are other finite values.
"""
import numpy as np
import pytest

from paged_kv_cache_pg_gb300 import pkv

from gpu_setup import torch

pytestmark = pytest.mark.gpu

HQ, HKV, IDX, STEPS, REPLAYS = 8, 2, 128, 24, 6
FMT = [pkv.KV_BF16, pkv.KV_E4M3]
KIND = ["decode", "window"]


@pytest.fixture(scope="module", autouse=True)
def built():
    from paged_kv_cache_pg_gb300 import build
    build.build()
    pkv.load()


class Chain:
    """Pages 0 .. n-1 and n .. 2n-1 of an arena hold the rows of two streams of
    T positions; `table` names the pages of one."""

    def __init__(self, fmt, kind, T, ptok, seed):
        t = torch()
        self.kind, self.T, self.ptok = kind, T, ptok
        self.lay = pkv.layout(1, HKV, 256, IDX, fmt)
        self.ps, self.n = pkv.page_elems(self.lay, ptok), -(-T // ptok)
        g = t.Generator(device="cuda").manual_seed(seed)
        self.rand = lambda *shape: t.randn(*shape, device="cuda", generator=g).to(t.bfloat16)
        self.mem = t.zeros(2 * self.n + 1, self.ps, dtype=t.int16, device="cuda")
        order = t.randperm(2 * self.n, device="cuda", generator=g).to(t.int32)
        self.ids = [order[:self.n].contiguous(), order[self.n:].contiguous()]
        self.table = self.ids[0].clone()
        self.rows = [[self.rand(T, HKV, 256), self.rand(T, HKV, 256), self.rand(T, IDX)] for _ in range(2)]
        for ids, rows in zip(self.ids, self.rows):
            pkv.store(self.lay, [pkv.seq(self.page(ids), T, T)], 0, *rows)
        self.first = self.mem.clone()
        self.status = t.zeros(1, dtype=t.int32, device="cuda")
        self.q, self.new = self.rand(STEPS, 1, HQ, 256), [self.rand(STEPS, 1, HKV, 256) for _ in range(2)] + [self.rand(STEPS, 1, IDX)]
        self.out = t.zeros_like(self.q)
        self.seen = t.zeros(STEPS, *self.mem.shape, dtype=t.int16, device="cuda")
        seqs = [pkv.seq(self.page(self.table), T, 1)]
        size = pkv.decode_ws_size(self.lay, seqs, HQ)
        self.ws = t.zeros(max(64, size // 4 + 64), dtype=t.float32, device="cuda")
        t.cuda.synchronize()

    def page(self, table):
        return pkv.pg(self.mem, table, self.ps, self.ptok, self.mem.shape[0], self.n)

    def decode(self, i, fused):
        seqs = [pkv.seq(self.page(self.table), self.T, 1)]
        k, v, ik = (x[i] for x in self.new) if fused else (None, None, None)
        if self.kind == "decode":
            pkv.decode(self.lay, seqs, 0, HQ, self.q[i], self.out[i], self.ws, status=self.status, k_new=k, v_new=v, ik_new=ik)
        else:
            pkv.window_decode(self.lay, seqs, 0, HQ, 2000, 4, self.q[i], self.out[i], None, status=self.status,
                              k_new=k, v_new=v, ik_new=ik)

    def check(self, reset, written, fused):
        """`reset`, then `written` and a decode right behind it, STEPS times."""
        t = torch()

        def step(i, wait):
            reset()
            for call in (written, lambda: self.decode(i, fused)):
                if wait:
                    t.cuda.synchronize()
                call()
            if wait:
                t.cuda.synchronize()
            self.seen[i].copy_(self.mem)

        for i in range(STEPS):
            step(i, True)
        t.cuda.synchronize()
        want = self.out.clone(), self.seen.clone()
        assert want[0].isfinite().all()
        graph = t.cuda.CUDAGraph()
        with t.cuda.graph(graph):
            for i in range(STEPS):
                step(i, False)
        for _ in range(REPLAYS):
            self.out.zero_()
            self.seen.zero_()
            graph.replay()
            t.cuda.synchronize()
            assert t.equal(self.out, want[0]) and t.equal(self.seen, want[1])
        assert int(self.status) == 0
        return want


@pytest.mark.parametrize("fmt", FMT)
@pytest.mark.parametrize("kind", KIND)
@pytest.mark.parametrize("T,ptok,tables", [(640, 16, 1), (600, 20, 4), (1024, 4, 2)])
def test_a_decode_behind_a_table_rewrite_uses_the_new_pages(T, ptok, tables, kind, fmt):
    t = torch()
    c = Chain(fmt, kind, T, ptok, 1)
    others = [c.ids[0].clone() for _ in range(tables - 1)]
    src, dst = (x.cpu().numpy() for x in c.ids)

    def reset():
        c.mem.copy_(c.first)
        for x in [c.table] + others:
            x.copy_(c.ids[0])

    out, seen = c.check(reset, lambda: pkv.tables_remap([c.table] + others, src, dst), fused=True)
    for i in range(STEPS):     # the new row went to the new page, the old pages are as they were
        changed = (seen[i] != c.first).any(1).nonzero().flatten().tolist()
        assert changed == [int(dst[(T - 1) // ptok])]


@pytest.mark.parametrize("fmt", FMT)
@pytest.mark.parametrize("kind", KIND)
@pytest.mark.parametrize("T,ptok,whole", [(1500, 64, True), (1003, 20, False)])
def test_a_decode_behind_page_copies_reads_the_copies(T, ptok, whole, kind, fmt):
    c = Chain(fmt, kind, T, ptok, 2)
    c.table.copy_(c.ids[1])
    src, dst = (x.cpu().numpy() for x in c.ids)
    n_pos = None if whole else np.array([min(ptok, T - ptok * j) for j in range(c.n)], np.int32)
    out, seen = c.check(lambda: c.mem.copy_(c.first),
                        lambda: pkv.pages_copy(c.lay, ptok, c.mem, c.mem.shape[0], src, dst, n_pos=n_pos), fused=False)
    c.table.copy_(c.ids[0])    # the first stream's own output
    c.mem.copy_(c.first)
    for i in range(STEPS):
        c.decode(i, False)
    assert torch().equal(c.out, out)


@pytest.mark.parametrize("fmt", FMT)
@pytest.mark.parametrize("kind", KIND)
@pytest.mark.parametrize("T,ptok", [(1500, 64), (333, 20)])
def test_a_decode_behind_a_store_reads_its_rows(T, ptok, kind, fmt):
    c = Chain(fmt, kind, T, ptok, 3)
    rows = [x[:T - 1].contiguous() for x in c.rows[1]]
    seq = [pkv.seq(c.page(c.table), T - 1, T - 1)]
    c.check(lambda: c.mem.copy_(c.first), lambda: pkv.store(c.lay, seq, 0, *rows, status=c.status), fused=True)
