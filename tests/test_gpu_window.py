"""Windowed decode on the GPU against the attention's definition in float64.

Rows that no query reads hold NaN bits and their pages' table entries are -1
in every case, so a key read out of its window shows.  The bound is the
framework's for float32-accumulated bf16 outputs (gpu_setup.bound): 1e-3 +
2e-3 |ref| and half a bf16 step.
"""
import numpy as np
import pytest

from paged_kv_cache_pg_gb300 import pkv, synth

from gpu_setup import GUARD, dev_u16, host_u16, torch, within_tol
from window_setup import Windowed, queries_of, streams_of

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    from paged_kv_cache_pg_gb300 import build
    build.build()
    pkv.load()


def run(w, layer, hq, q_list, fused=False, expect=0, stream=None):
    t = torch()
    seqs = w.seqs()
    q = dev_u16(np.concatenate(q_list))
    out = t.full_like(q, 0x7FC1)
    size = pkv.window_decode_ws_size(w.lay, seqs, hq, w.window, w.sinks)
    ws = t.full((max(64, size // 4),), float("nan"), dtype=t.float32, device="cuda") if size else None
    status = t.zeros(1, dtype=t.int32, device="cuda")
    k, v, ik = w.new_rows(layer) if fused else (None, None, None)
    pkv.window_decode(w.lay, seqs, layer, hq, w.window, w.sinks, q, out, ws, status=status, k_new=k, v_new=v, ik_new=ik)
    t.cuda.synchronize()
    assert int(status.item()) == expect
    return host_u16(out)


FMT = [pkv.KV_BF16, pkv.KV_E4M3]
# (lens, n_new, hq, hkv, window, sinks)
SHAPES = [
    ([1], [1], 4, 1, 1, 0),                                # one token
    ([1, 2, 40], [1, 2, 3], 8, 2, 2, 1),                   # more new tokens than the window
    ([300], [1], 4, 1, 128, 4),
    ([300, 17, 64, 65], [1, 1, 1, 1], 16, 2, 16, 0),       # windows of one tile, tile borders
    ([100, 500, 333], [1, 4, 2], 16, 2, 100, 17),          # ragged new tokens, 32 columns
    ([200, 230], [1, 2], 6, 2, 50, 64),                    # groups of 3, sinks past a tile
    ([90, 120], [3, 1], 5, 1, 100, 99),                    # sinks and window meet
    ([150, 31], [1, 1], 3, 3, 500, 7),                     # windows longer than the streams
    ([700], [1], 32, 1, 300, 300),                         # 32 heads of one KV head
    ([1500, 900], [1, 1], 8, 8, 1000, 1000),               # sinks as long as the window
    ([130, 66], [1, 3], 8, 2, 100, 18),                    # small pages gone inside one tile
    ([400, 0, 77], [1, 0, 1], 16, 2, 60, 5),               # a stream without queries, an empty one
]


@pytest.mark.parametrize("fmt", FMT)
@pytest.mark.parametrize("ptok", [4, 20, 16, 256, None])
@pytest.mark.parametrize("case", range(len(SHAPES)))
def test_decode_matches_the_definition(case, ptok, fmt):
    lens, n_new, hq, hkv, window, sinks = SHAPES[case]
    lay = pkv.layout(1, hkv, 256, 0, fmt)
    w = Windowed(lay, streams_of(lens, hkv, seed=10 * case), n_new, window, sinks, ptok, seed=case)
    q = queries_of(n_new, hq, seed=case)
    ok, report = within_tol(run(w, 0, hq, q), w.reference(0, q))
    assert ok, report


@pytest.mark.parametrize("fmt", FMT)
@pytest.mark.parametrize("ptok", [20, 128])
def test_long_windows_are_split_and_combined(fmt, ptok):
    # 9,000 keys of a stream: two splits of eight CTAs; the short stream has one
    lens, n_new, hq, hkv, window, sinks = [12000, 300, 9500], [1, 1, 2], 8, 2, 9000, 33
    lay = pkv.layout(1, hkv, 256, 0, fmt)
    w = Windowed(lay, streams_of(lens, hkv, seed=7), n_new, window, sinks, ptok, seed=3)
    q = queries_of(n_new, hq, seed=5)
    got = run(w, 0, hq, q)
    ok, report = within_tol(got, w.reference(0, q))
    assert ok, report
    c = Windowed(lay, w.streams, n_new, window, sinks, None)
    assert np.array_equal(run(c, 0, hq, q), got)


@pytest.mark.parametrize("fmt", FMT)
def test_a_full_launch_of_ragged_streams(fmt):
    # 1,024 CTAs in clusters of eight, several waves, streams of 1 to 2,800 positions
    lens = [1 + (i * 1733) % 2800 for i in range(64)]
    n_new, hq, hkv, window, sinks = [1] * 64, 4, 2, 2000, 4
    lay = pkv.layout(1, hkv, 256, 128, fmt)
    w = Windowed(lay, streams_of(lens, hkv, 128, seed=70), n_new, window, sinks, 64, seed=2, fused=True)
    q = queries_of(n_new, hq, seed=70)
    want = w.reference(0, q)
    for _ in range(3):
        ok, report = within_tol(run(w, 0, hq, q, fused=True), want)
        assert ok, report


@pytest.mark.parametrize("fmt", FMT)
def test_full_launches_back_to_back_give_the_same_bits(fmt):
    # 64 streams of 4,100-key windows: 33 tiles a CTA go several times around
    # its stages while the memory is saturated and tiles land out of order
    t = torch()
    B, T, hq, hkv, ptok = 64, 4500, 16, 2, 64
    lay = pkv.layout(1, hkv, 256, 0, fmt)
    ps, per = pkv.page_elems(lay, ptok), synth.pages_for(T, ptok)
    mem = t.zeros(B * per, ps, dtype=t.int16, device="cuda")
    table = t.randperm(B * per, device="cuda").to(t.int32).view(B, per)
    seqs = pkv.batch([pkv.seq(pkv.pg(mem, table[i], ps, ptok, B * per), T - i, 1) for i in range(B)])
    rows = t.randn(T, hkv, 256, device="cuda").to(t.bfloat16)
    for i in range(B):
        pkv.store(lay, [pkv.seq(seqs[i].pg, T, T)], 0, rows.roll(i, 0).contiguous(), rows.roll(-i, 0).contiguous())
    q = t.randn(B, hq, 256, device="cuda").to(t.bfloat16)
    status = t.zeros(1, dtype=t.int32, device="cuda")
    outs = [t.zeros_like(q) for _ in range(40)]
    ws = t.empty(pkv.window_decode_ws_size(lay, seqs, hq, 4096, 4) // 4, dtype=t.float32, device="cuda")
    for o in outs:
        pkv.window_decode(lay, seqs, 0, hq, 4096, 4, q, o, ws, status=status)
    assert int(status) == 0 and outs[0].isfinite().all()
    assert all(t.equal(o, outs[0]) for o in outs)
    # a stream alone takes the clustered kernel, the batch the combine: the same bits
    assert ws.numel() > 0
    for i in (0, 17, 63):
        alone = t.zeros_like(q[i:i + 1])
        assert pkv.window_decode_ws_size(lay, seqs[i:i + 1], hq, 4096, 4) == 0
        pkv.window_decode(lay, seqs[i:i + 1], 0, hq, 4096, 4, q[i:i + 1], alone)
        assert t.equal(alone, outs[0][i:i + 1])


@pytest.mark.parametrize("fmt", FMT)
def test_paged_equals_contiguous_and_alone_equals_in_batch(fmt):
    lens, n_new, hq, hkv, window, sinks = [1000, 77, 2500, 640], [1, 2, 1, 2], 16, 2, 512, 4
    lay = pkv.layout(1, hkv, 256, 0, fmt)
    streams = streams_of(lens, hkv, seed=31)
    q = queries_of(n_new, hq, seed=31)
    base = run(Windowed(lay, streams, n_new, window, sinks, None), 0, hq, q)
    for ptok in (4, 16, 20, 48, 256):
        assert np.array_equal(run(Windowed(lay, streams, n_new, window, sinks, ptok, seed=ptok), 0, hq, q), base)
    rows = np.split(base, np.cumsum(n_new)[:-1])
    for i in range(4):
        w = Windowed(lay, streams[i:i + 1], n_new[i:i + 1], window, sinks, 48, seed=i)
        assert np.array_equal(run(w, 0, hq, q[i:i + 1]), rows[i])


# (lens, new tokens, q heads, kv heads, window, sinks, indexer dim) of calls that
# give a KV head's 17 to 32 query columns one CTA: several pieces, splits, one
# piece; the last one's columns are two CTAs
WIDE = [([int(x) for x in np.linspace(40, 2300, 24)], [4, 3, 2, 1] * 6, 16, 2, 1500, 4, 128),
        ([9100, 8000, 9005, 7000, 8800, 9216, 8191, 30], [4, 4, 3, 4, 1, 4, 4, 4], 16, 2, 9000, 0, 0),
        ([int(x) for x in np.linspace(5, 200, 64)], [4, 3, 0, 2] * 16, 32, 4, 60, 1, 0),
        ([700, 37, 150], [4, 3, 4], 16, 2, 300, 5, 128)]


@pytest.mark.parametrize("fmt", FMT)
@pytest.mark.parametrize("case", range(len(WIDE)))
def test_many_draft_windows(case, fmt):
    t = torch()
    lens, n_new, hq, hkv, window, sinks, idx = WIDE[case]
    lay = pkv.layout(1, hkv, 256, idx, fmt)
    streams = streams_of(lens, hkv, idx, seed=400)
    q = queries_of(n_new, hq, seed=400)
    a = Windowed(lay, streams, n_new, window, sinks, 48, seed=1, fused=True)
    b = Windowed(lay, streams, n_new, window, sinks, 48, seed=1, fused=True)
    pkv.store(lay, b.seqs(), 0, *b.new_rows(0))
    got = run(a, 0, hq, q, fused=True)
    assert np.array_equal(got, run(b, 0, hq, q))
    assert t.equal(a.bufs[0], b.bufs[0])
    rows = np.split(got, np.cumsum(n_new)[:-1])
    for i in sorted({0, 1, 2, 3, 5, len(lens) - 1}):
        if i >= len(lens) or n_new[i] == 0:
            continue
        w = Windowed(lay, streams[i:i + 1], n_new[i:i + 1], window, sinks, 16, seed=i)
        ok, report = within_tol(rows[i], w.reference(0, q[i:i + 1]))
        assert ok, report
        assert np.array_equal(run(w, 0, hq, q[i:i + 1]), rows[i])   # alone, a CTA takes 16 columns


@pytest.mark.parametrize("fmt", FMT)
@pytest.mark.parametrize("ptok", [16, 20, 64])
@pytest.mark.parametrize("idx", [0, 128])
def test_the_call_stores_its_new_rows(fmt, ptok, idx):
    t = torch()
    lens, n_new, hq, hkv, window, sinks, layer = [130, 16, 77], [2, 3, 1], 8, 2, 40, 4, 1
    lay = pkv.layout(2, hkv, 256, idx, fmt)
    streams = streams_of(lens, hkv, idx, layers=2, seed=50)
    q = queries_of(n_new, hq, seed=50)
    a = Windowed(lay, streams, n_new, window, sinks, ptok, seed=1, fused=True)
    b = Windowed(lay, streams, n_new, window, sinks, ptok, seed=1, fused=True)
    k, v, ik = b.new_rows(layer)
    pkv.store(lay, b.seqs(), layer, k, v, ik)
    got = run(a, layer, hq, q, fused=True)
    ok, report = within_tol(got, a.reference(layer, q))
    assert ok, report
    assert np.array_equal(got, run(b, layer, hq, q))                    # as a store and a decode
    assert t.equal(a.bufs[0], b.bufs[0])                                # the same bytes, guards and all


def test_a_row_that_is_read_behind_a_bad_page_is_reported():
    t = torch()
    lay = pkv.layout(1, 1, 256, 0)
    w = Windowed(lay, streams_of([200], 1), [1], 64, 4, 16)
    q = queries_of([1], 4)
    run(w, 0, 4, q)                                                     # the pages behind the window are not looked at
    w.pgs[0].n_table = 13
    table = next(x for x in w.keep if x.dtype == t.int32)
    table[12] = 1 << 20
    run(w, 0, 4, q, expect=pkv.DEV_BAD_PAGE)
    table[12] = -7
    run(w, 0, 4, q, expect=pkv.DEV_BAD_PAGE)


def test_one_arena_beyond_four_gigabytes():
    # pages at byte offsets past 2^32: the stream's pages are the last of a 4.9 GB arena
    t = torch()
    lay = pkv.layout(1, 2, 256, 0)
    w = Windowed(lay, streams_of([700], 2), [1], 300, 4, 64, seed=1)
    q = queries_of([1], 8)
    want = run(w, 0, 8, q)
    ps = pkv.page_elems(lay, 64)
    small = w._body(0)
    n = small.numel() // ps
    total = 4_900_000_000 // (2 * ps)
    big = t.zeros(total * ps, dtype=t.int16, device="cuda")
    big[-small.numel():] = small
    table = next(x for x in w.keep if x.dtype == t.int32)
    moved = t.where(table >= 0, table + (total - n), table)
    w.pgs[0] = pkv.pg(big, moved, ps, 64, total, table.numel() - 1)
    assert np.array_equal(run(w, 0, 8, q), want)


def test_captured_and_replayed_with_new_inputs_on_another_stream():
    t = torch()
    lens, n_new, hq, window, sinks = [9000, 8200], [1, 1], 8, 6000, 4   # with a workspace
    lay = pkv.layout(1, 1, 256, 0)
    w = Windowed(lay, streams_of(lens, 1, seed=3), n_new, window, sinks, 64)
    qs = [queries_of(n_new, hq, seed=s) for s in (1, 2)]
    want = [run(w, 0, hq, q) for q in qs]
    seqs = pkv.batch(w.seqs())
    q = dev_u16(np.concatenate(qs[0]))
    size = pkv.window_decode_ws_size(lay, seqs, hq, window, sinks) // 4
    assert size > 0
    # two graphs that share a workspace, replayed in order
    ws = t.empty(size, dtype=t.float32, device="cuda")
    outs, graphs = [t.zeros_like(q) for _ in range(2)], []
    for o in outs:
        g = t.cuda.CUDAGraph()
        with t.cuda.graph(g):
            pkv.window_decode(lay, seqs, 0, hq, window, sinks, q, o, ws)
        graphs.append(g)
    side = t.cuda.Stream()
    side.wait_stream(t.cuda.current_stream())
    with t.cuda.stream(side):
        for i in (0, 1, 0):
            q.copy_(dev_u16(np.concatenate(qs[i])))
            for g in graphs:
                g.replay()
            side.synchronize()
            assert all(np.array_equal(host_u16(o), want[i]) for o in outs)


def test_token_by_token_with_pages_given_back():
    """A stream decodes past its window, giving dead pages back to the arena:
    they are taken again and overwritten, and every step agrees with the
    definition."""
    t = torch()
    hq, hkv, window, sinks, ptok, start, steps = 4, 1, 40, 5, 16, 60, 120
    lay = pkv.layout(1, hkv, 256, 0)
    s = synth.make_stream(9, 1, start + steps, hkv, 256, 0)
    ps = pkv.page_elems(lay, ptok)
    n_pages = 6                                       # far fewer than the stream's 12 pages
    mem = t.full((n_pages * ps,), 0x7FC1, dtype=t.int16, device="cuda")
    a = pkv.Arena(lay, ptok, mem)
    ids = list(a.take(4))
    table = t.full((12,), -1, dtype=t.int32, device="cuda")
    table[:4] = t.tensor(ids, dtype=t.int32)
    g = a.pg(table)
    status = t.zeros(1, dtype=t.int32, device="cuda")
    pkv.store(lay, [pkv.seq(g, start, start)], 0, dev_u16(s.k[0][:start]), dev_u16(s.v[0][:start]))
    k, v, dead = dev_u16(s.k[0]), dev_u16(s.v[0]), 0
    outs, qs = [], []
    for n in range(start + 1, start + steps + 1):
        first, end = pkv.window_dead_pages(ptok, n - 1, window, sinks)
        for p in range(max(first, dead), end):
            a.give([ids[p]])
            t.cuda.synchronize()
            mem.view(n_pages, ps)[int(ids[p])] = 0x7FC1
            table[p], dead = -1, p + 1
        if (n - 1) // ptok == len(ids):
            ids.append(int(a.take(1)[0]))
            table[len(ids) - 1] = ids[-1]
        qs.append(synth.queries(n, 1, hq, 256))
        q = dev_u16(qs[-1])
        out = t.zeros_like(q)
        pkv.window_decode(lay, [pkv.seq(g, n, 1)], 0, hq, window, sinks, q, out, status=status,
                          k_new=k[n - 1:n], v_new=v[n - 1:n])
        outs.append(out)
    from window_setup import attend, values
    kf, vf = values(s.k[0], lay.kv_format), values(s.v[0], lay.kv_format)
    for i, (o, q) in enumerate(zip(outs, qs)):
        ok, report = within_tol(host_u16(o), attend(kf, vf, q, start + 1 + i, window, sinks))
        assert ok, (i, report)
    assert int(status) == 0 and dead >= 7


@pytest.mark.parametrize("fmt", FMT)
def test_calls_of_32_tokens_follow_each_other_directly(fmt):
    # each call stores 32 rows, and the next reads cached rows more than 32 below
    # its own new ones before the call has finished
    t = torch()
    T, hkv, ptok, steps = 1024, 2, 16, 32
    lay = pkv.layout(1, hkv, 256, 0, fmt)
    ps, per = pkv.page_elems(lay, ptok), T // ptok
    g = t.Generator(device="cuda").manual_seed(5)
    table = t.randperm(per, device="cuda", generator=g).to(t.int32)
    k, v, q = (t.randn(T, hkv, 256, device="cuda", generator=g).to(t.bfloat16) for _ in range(3))
    outs = []
    for wait in (True, False):
        mem = t.full((per, ps), 0x7FC1, dtype=t.int16, device="cuda")
        out = t.zeros_like(q)
        status = t.zeros(1, dtype=t.int32, device="cuda")
        calls = []
        for i in range(steps):
            at = slice(32 * i, 32 * i + 32)
            seqs = pkv.batch([pkv.seq(pkv.pg(mem, table, ps, ptok, per), 32 * i + 32, 32)])
            calls.append((seqs, q[at].contiguous(), out[at], k[at].contiguous(), v[at].contiguous()))
        t.cuda.synchronize()

        def run_all():
            for seqs, qi, oi, ki, vi in calls:
                pkv.window_decode(lay, seqs, 0, hkv, 200, 4, qi, oi, None, status=status, k_new=ki, v_new=vi)
                if wait:
                    t.cuda.synchronize()

        if wait:
            run_all()
        else:
            graph = t.cuda.CUDAGraph()
            with t.cuda.graph(graph):
                run_all()
            for _ in range(5):
                mem.fill_(0x7FC1)
                out.zero_()
                graph.replay()
        t.cuda.synchronize()
        assert int(status) == 0
        outs.append((out.clone(), mem))
    assert t.equal(outs[0][0], outs[1][0]) and t.equal(outs[0][1], outs[1][1])
    assert outs[0][0].isfinite().all()


@pytest.mark.parametrize("fmt", FMT)
def test_more_contiguous_streams_than_copy_maps(fmt):
    lens, hq, hkv, window, sinks = [int(x) for x in np.linspace(3, 700, 40)], 16, 2, 300, 4
    lay = pkv.layout(1, hkv, 256, 0, fmt)
    streams = streams_of(lens, hkv, seed=500)
    q = queries_of([1] * 40, hq, seed=500)
    a = Windowed(lay, streams, [1] * 40, window, sinks, None)
    b = Windowed(lay, streams, [1] * 40, window, sinks, 32, seed=3)
    got = run(a, 0, hq, q)
    ok, report = within_tol(got, a.reference(0, q))
    assert ok, report
    assert np.array_equal(got, run(b, 0, hq, q))


@pytest.mark.parametrize("fmt", FMT)
@pytest.mark.parametrize("streams", [2, 24])
def test_output_rows_behind_the_last_stream_stay(fmt, streams):
    t = torch()
    lens, hq, hkv, window, sinks = [200 + i for i in range(streams)], 16, 2, 1100, 4
    lay = pkv.layout(1, hkv, 256, 0, fmt)
    w = Windowed(lay, streams_of(lens, hkv, seed=600), [3] * streams, window, sinks, 16)
    seqs, rows = w.seqs(), 3 * streams
    q = dev_u16(np.concatenate(queries_of([3] * streams, hq, seed=600)))
    out = t.full((rows + 5, hq, 256), 0x7FC1, dtype=q.dtype, device="cuda")
    size = pkv.window_decode_ws_size(lay, seqs, hq, window, sinks)
    ws = t.full((size // 4 + 64,), 7.5, dtype=t.float32, device="cuda")
    pkv.window_decode(lay, seqs, 0, hq, window, sinks, q, out, ws)
    assert (out[rows:] == 0x7FC1).all() and (ws[size // 4:] == 7.5).all()
    assert not (out[:rows] == 0x7FC1).any()
