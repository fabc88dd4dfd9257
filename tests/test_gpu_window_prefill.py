"""Windowed chunk attention on the GPU against the attention's definition in
float64.  As in the decode's tests, rows that no query reads hold NaN bits and
their pages' table entries are -1.  Bound: gpu_setup.bound."""
import numpy as np
import pytest

import oracle as orc
from paged_kv_cache_pg_gb300 import pkv, synth

from gpu_setup import dev_u16, host_u16, torch, within_tol
from window_setup import Windowed, attend, queries_of, streams_of, values

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    from paged_kv_cache_pg_gb300 import build
    build.build()
    pkv.load()


def workspace(lay, seqs, hq, window, sinks):
    t = torch()
    size = pkv.window_prefill_ws_size(lay, seqs, hq, window, sinks)
    return t.full((max(64, size // 4),), float("nan"), dtype=t.float32, device="cuda")


def run(w, layer, hq, q_list, expect=0):
    t = torch()
    seqs = w.seqs()
    q = dev_u16(np.concatenate(q_list))
    out = t.full_like(q, 0x7FC1)
    status = t.zeros(1, dtype=t.int32, device="cuda")
    pkv.window_prefill(w.lay, seqs, layer, hq, w.window, w.sinks, q, out, workspace(w.lay, seqs, hq, w.window, w.sinks),
                       status=status)
    t.cuda.synchronize()
    assert int(status.item()) == expect
    return host_u16(out)


# (lens, n_new, hq, hkv, window, sinks)
SHAPES = [
    ([1], [1], 4, 1, 1, 0),
    ([90], [90], 8, 1, 16, 4),                       # a prompt from its start
    ([300, 64], [40, 64], 16, 2, 100, 4),            # ragged streams, rows that end inside an M-tile
    ([260], [33], 5, 1, 40, 18),                     # groups of 5; small pages gone inside one run
    ([200, 3], [17, 3], 6, 2, 500, 7),               # windows longer than the streams
    ([400], [200], 3, 3, 128, 130),                  # a head a group, sinks over a tile
    ([640], [64], 16, 1, 200, 300),                  # sinks meet the window
    ([333, 0, 50], [100, 0, 1], 8, 2, 1, 1),         # a window of one, a stream without queries
    ([1100], [20], 4, 1, 900, 70),                   # few rows: splits
    ([700, 650], [300, 5], 8, 4, 256, 16),
]


@pytest.mark.parametrize("ptok", [4, 20, 16, 256, None])
@pytest.mark.parametrize("case", range(len(SHAPES)))
def test_chunk_matches_the_definition(case, ptok):
    lens, n_new, hq, hkv, window, sinks = SHAPES[case]
    lay = pkv.layout(1, hkv, 256, 0)
    w = Windowed(lay, streams_of(lens, hkv, seed=10 * case), n_new, window, sinks, ptok, seed=case)
    q = queries_of(n_new, hq, seed=case)
    ok, report = within_tol(run(w, 0, hq, q), w.reference(0, q))
    assert ok, report


def test_paged_equals_contiguous_and_alone_equals_in_batch():
    lens, n_new, hq, hkv, window, sinks = [1000, 77, 2500], [300, 77, 9], 16, 2, 512, 4
    lay = pkv.layout(1, hkv, 256, 0)
    streams = streams_of(lens, hkv, seed=31)
    q = queries_of(n_new, hq, seed=31)
    base = run(Windowed(lay, streams, n_new, window, sinks, None), 0, hq, q)
    for ptok in (4, 16, 20, 48, 256):
        assert np.array_equal(run(Windowed(lay, streams, n_new, window, sinks, ptok, seed=ptok), 0, hq, q), base)
    rows = np.split(base, np.cumsum(n_new)[:-1])
    for i in range(3):
        w = Windowed(lay, streams[i:i + 1], n_new[i:i + 1], window, sinks, 48, seed=i)
        assert np.array_equal(run(w, 0, hq, q[i:i + 1]), rows[i])


def _sampled(w, q_list, got, picks):
    """Rows (stream, query) of the output against the definition."""
    at = np.cumsum([0] + w.n_new)
    for s, j in picks:
        st = w.streams[s]
        p = st.length - w.n_new[s] + j
        k, v = values(st.k[0][:p + 1], w.lay.kv_format), values(st.v[0][:p + 1], w.lay.kv_format)
        ok, report = within_tol(got[at[s] + j:at[s] + j + 1], attend(k, v, q_list[s][j:j + 1], p + 1, w.window, w.sinks))
        assert ok, (s, j, report)


@pytest.mark.parametrize("hq,hkv,lens,n_new,window,sinks", [
    (8, 8, [2600, 2500], [2600, 700], 300, 4),       # 208 items and more: several a CTA
    (16, 2, [6000], [4100], 777, 20),                # 514 M-tiles over two KV heads
    (4, 1, [20000], [700], 9000, 4),                 # long windows, few M-tiles: splits
])
def test_long_chunks_on_sampled_rows(hq, hkv, lens, n_new, window, sinks):
    lay = pkv.layout(1, hkv, 256, 0)
    w = Windowed(lay, streams_of(lens, hkv, seed=90), n_new, window, sinks, 64, seed=4)
    q = queries_of(n_new, hq, seed=90)
    got = run(w, 0, hq, q)
    assert np.isfinite(orc.bf16_to_float(got)).all()
    rng = np.random.default_rng(8)
    for s in range(len(lens)):
        _sampled(w, q, got, [(s, j) for j in {0, n_new[s] - 1, 16, *rng.integers(0, n_new[s], 25).tolist()}])
    again = run(w, 0, hq, q)
    assert np.array_equal(got, again)


def test_maxima_that_grow_along_the_keys_rescale():
    # keys that grow by steps along the context, queries along them: the
    # running maximum passes the lazy rescale's threshold several times a row
    lay = pkv.layout(1, 1, 256, 0)
    s = streams_of([1200], 1, seed=5)[0]
    d = synth.normal_bf16(1, (256,))
    f = (np.arange(1200) // 130 + 1).astype(np.float32)[:, None, None] * 0.25
    k = (orc.bf16_to_float(d)[None, None] * f).astype(np.float32)
    s.k[0] = (k.view(np.uint32) >> 16).astype(np.uint16)
    w = Windowed(lay, [s], [60], 1000, 4, 16)
    q = [np.broadcast_to(d, (60, 4, 256)).copy()]
    ok, report = within_tol(run(w, 0, 4, q), w.reference(0, q))
    assert ok, report


def test_v_beyond_fp16_is_reported_and_the_largest_is_exact():
    lay = pkv.layout(1, 1, 256, 0)
    s = streams_of([100], 1, seed=6)[0]
    s.v[0][50, 0, 7] = 0x477F                        # 65,280, bf16's last value in fp16's range
    q = queries_of([50], 4)
    w = Windowed(lay, [s], [50], 60, 4, 16)
    ok, report = within_tol(run(w, 0, 4, q), w.reference(0, q))
    assert ok, report
    s.v[0][50, 0, 7] = 0x4780                        # 65,536
    run(Windowed(lay, [s], [50], 60, 4, 16), 0, 4, q, expect=pkv.DEV_RANGE)


def test_a_row_that_is_read_behind_a_bad_page_is_reported():
    t = torch()
    lay = pkv.layout(1, 1, 256, 0)
    w = Windowed(lay, streams_of([200], 1), [20], 64, 4, 16)
    q = queries_of([20], 4)
    run(w, 0, 4, q)
    table = next(x for x in w.keep if x.dtype == t.int32)
    table[12] = 1 << 20
    # page 0 is read instead, which holds NaN here: reported too
    run(w, 0, 4, q, expect=pkv.DEV_BAD_PAGE | pkv.DEV_RANGE)


def test_captured_graphs_share_a_workspace_and_replay_with_new_inputs():
    t = torch()
    lens, n_new, hq, window, sinks = [1500, 900], [200, 30], 8, 700, 4
    lay = pkv.layout(1, 1, 256, 0)
    w = Windowed(lay, streams_of(lens, 1, seed=3), n_new, window, sinks, 64)
    qs = [queries_of(n_new, hq, seed=s) for s in (1, 2)]
    want = [run(w, 0, hq, q) for q in qs]
    seqs = pkv.batch(w.seqs())
    q = dev_u16(np.concatenate(qs[0]))
    ws = workspace(lay, seqs, hq, window, sinks)
    outs, graphs = [t.zeros_like(q) for _ in range(2)], []
    for o in outs:
        g = t.cuda.CUDAGraph()
        with t.cuda.graph(g):
            pkv.window_prefill(lay, seqs, 0, hq, window, sinks, q, o, ws)
        graphs.append(g)
    for i in (0, 1, 0):
        q.copy_(dev_u16(np.concatenate(qs[i])))
        for g in graphs:
            g.replay()
        t.cuda.synchronize()
        assert all(np.array_equal(host_u16(o), want[i]) for o in outs)


def test_back_to_back_calls_give_the_same_bits():
    t = torch()
    lens, n_new, hq, hkv, window, sinks = [3000, 1000, 500], [1500, 1000, 33], 16, 2, 400, 4
    lay = pkv.layout(1, hkv, 256, 0)
    w = Windowed(lay, streams_of(lens, hkv, seed=13), n_new, window, sinks, 64)
    q = dev_u16(np.concatenate(queries_of(n_new, hq, seed=1)))
    seqs = pkv.batch(w.seqs())
    ws, status = workspace(lay, seqs, hq, window, sinks), t.zeros(1, dtype=t.int32, device="cuda")
    outs = [t.zeros_like(q) for _ in range(60)]
    for o in outs:
        pkv.window_prefill(lay, seqs, 0, hq, window, sinks, q, o, ws, status=status)
    assert int(status) == 0
    assert all(t.equal(o, outs[0]) for o in outs)


def test_prompt_in_chunks_then_tokens_in_a_small_arena():
    """A prompt stored and attended in chunks, dead pages given back after
    each, then decoded token by token, in an arena that could not hold it
    whole; layer 1 of 2."""
    t = torch()
    hq, hkv, window, sinks, ptok, layer = 8, 2, 90, 6, 16, 1
    lay = pkv.layout(2, hkv, 256, 128)
    T, tail = 500, 12
    s = synth.make_stream(4, 2, T + tail, hkv, 256, 128)
    ps = pkv.page_elems(lay, ptok)
    n_pages = 15                                     # of the 32 that the stream goes through
    mem = t.full((n_pages * ps,), 0x7FC1, dtype=t.int16, device="cuda")
    a = pkv.Arena(lay, ptok, mem)
    table = t.full((synth.pages_for(T + tail, ptok),), -1, dtype=t.int32, device="cuda")
    g, ids, dead = a.pg(table), [], 0
    status = t.zeros(1, dtype=t.int32, device="cuda")
    kf, vf = values(s.k[layer], 0), values(s.v[layer], 0)
    rng, at, step = np.random.default_rng(1), 0, 0
    while at < T + tail:
        n = min(int(rng.integers(1, 110)), T - at) if at < T else 1
        first, end = pkv.window_dead_pages(ptok, at, window, sinks)
        gone = [p for p in range(max(first, dead), end)]
        if gone:
            a.give([ids[p] for p in gone])
            t.cuda.synchronize()
            for p in gone:
                mem.view(n_pages, ps)[int(ids[p])] = 0x7FC1
                table[p] = -1
            dead = end
        need = synth.pages_for(at + n, ptok) - len(ids)
        for i in a.take(need):
            table[len(ids)] = int(i)
            ids.append(i)
        sq = [pkv.seq(g, at + n, n)]
        rows = [dev_u16(x[layer][at:at + n]) for x in (s.k, s.v, s.ik)]
        qb = synth.queries(step, n, hq, 256)
        q = dev_u16(qb)
        out = t.zeros_like(q)
        if at < T:
            pkv.store(lay, sq, layer, *rows, status=status)
            pkv.pool(lay, sq, layer, status=status)
            pkv.window_prefill(lay, sq, layer, hq, window, sinks, q, out, workspace(lay, sq, hq, window, sinks), status=status)
        else:
            pkv.window_decode(lay, sq, layer, hq, window, sinks, q, out, status=status, k_new=rows[0], v_new=rows[1],
                              ik_new=rows[2])
        ok, report = within_tol(host_u16(out), attend(kf, vf, qb, at + n, window, sinks))
        assert ok, (at, n, report)
        at, step = at + n, step + 1
    assert int(status) == 0 and dead > 20


@pytest.mark.parametrize("lens,n_new,window", [([300, 64], [40, 64], 100), ([1100], [20], 900)])
def test_output_rows_behind_the_last_stream_stay(lens, n_new, window):
    t = torch()
    hq, hkv, sinks, rows = 8, 2, 4, sum(n_new)
    lay = pkv.layout(1, hkv, 256, 0)
    w = Windowed(lay, streams_of(lens, hkv, seed=700), n_new, window, sinks, 20)
    seqs = w.seqs()
    q = dev_u16(np.concatenate(queries_of(n_new, hq, seed=700)))
    out = t.full((rows + 200, hq, 256), 0x7FC1, dtype=q.dtype, device="cuda")
    size = pkv.window_prefill_ws_size(lay, seqs, hq, window, sinks)
    ws = t.full((size // 4 + 64,), 7.5, dtype=t.float32, device="cuda")
    pkv.window_prefill(lay, seqs, 0, hq, window, sinks, q, out, ws)
    assert (out[rows:] == 0x7FC1).all() and (ws[size // 4:] == 7.5).all()
    assert not (out[:rows] == 0x7FC1).any()


def test_calls_on_two_streams_at_once():
    # a chunk and decodes on one stream, the same with other inputs on a second: each
    # with its own workspaces, and the results of running them one after the other
    t = torch()
    hq, hkv, window, sinks = 16, 2, 512, 4
    lay = pkv.layout(1, hkv, 256, 0)
    sets = []
    for k in range(2):
        dec = Windowed(lay, streams_of([600 + 7 * i for i in range(24)], hkv, seed=800 + 40 * k), [1] * 24, window, sinks, 16)
        pre = Windowed(lay, streams_of([900, 333], hkv, seed=880 + k), [256, 100], window, sinks, 16)
        dq, pq = (dev_u16(np.concatenate(queries_of(w.n_new, hq, seed=900 + k))) for w in (dec, pre))
        dseq, pseq = pkv.batch(dec.seqs()), pkv.batch(pre.seqs())
        size = pkv.window_decode_ws_size(lay, dseq, hq, window, sinks)
        dws = t.empty(max(64, size // 4), dtype=t.float32, device="cuda")
        sets.append((dec, pre, dq, pq, dseq, pseq, dws, workspace(lay, pseq, hq, window, sinks)))

    def calls(k, stream):
        _, _, dq, pq, dseq, pseq, dws, pws = sets[k]
        outs = []
        for _ in range(12):
            outs += [t.zeros_like(dq), t.zeros_like(pq)]
            stream.wait_stream(t.cuda.default_stream())
            pkv.window_decode(lay, dseq, 0, hq, window, sinks, dq, outs[-2], dws, stream=stream)
            pkv.window_prefill(lay, pseq, 0, hq, window, sinks, pq, outs[-1], pws, stream=stream)
        return outs

    alone = []
    for k in range(2):
        alone.append(calls(k, t.cuda.default_stream()))
        t.cuda.synchronize()
    side = [t.cuda.Stream(), t.cuda.Stream()]
    both = [calls(k, side[k]) for k in range(2)]
    t.cuda.synchronize()
    for k in range(2):
        assert all(t.equal(x, alone[k][i % 2]) for i, x in enumerate(alone[k] + both[k]))
