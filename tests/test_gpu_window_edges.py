"""Windowed decode at the edges of its plan and of its inputs' range, against the
attention's definition in float64 (bound: gpu_setup.bound)."""
import numpy as np
import pytest

from paged_kv_cache_pg_gb300 import pkv, synth

from gpu_setup import dev_u16, host_u16, torch, within_tol
from window_setup import Windowed, attend, queries_of, streams_of, values

pytestmark = pytest.mark.gpu

FMT = [pkv.KV_BF16, pkv.KV_E4M3]


@pytest.fixture(scope="module", autouse=True)
def built():
    from paged_kv_cache_pg_gb300 import build
    build.build()
    pkv.load()


@pytest.mark.parametrize("fmt", FMT)
def test_one_workspace_for_every_length_near_a_split_s_border(fmt):
    t = torch()
    hq, hkv, sinks = 8, 1, 4
    window = 5106 if fmt == pkv.KV_BF16 else 5090
    lay = pkv.layout(1, hkv, 256, 0, fmt)
    longest = streams_of([5400], hkv, seed=41)[0]
    top = pkv.pg(1 << 20, None, pkv.page_elems(lay, 20000), 20000)
    size = pkv.window_decode_ws_size(lay, [pkv.seq(top, 20000, 2)], hq, window, sinks)
    ws = t.full((size // 4 + 64,), float("nan"), dtype=t.float32, device="cuda")
    status = t.zeros(1, dtype=t.int32, device="cuda")
    for n in [60, window - 20, window, *range(5180, 5218, 5), 5400]:
        s = synth.Stream(n, longest.k, longest.v, longest.ik)
        w = Windowed(lay, [s], [2], window, sinks, 64, seed=n)
        q = queries_of([2], hq, seed=n)
        out = t.full((2, hq, 256), 0x7FC1, dtype=t.int16, device="cuda")
        pkv.window_decode(lay, w.seqs(), 0, hq, window, sinks, dev_u16(q[0]), out, ws[:size // 4], status=status)
        ok, report = within_tol(host_u16(out), w.reference(0, q))
        assert ok, (n, report)
    assert int(status) == 0 and ws[size // 4:].isnan().all()



def run(w, hq, q_list, **new):
    t = torch()
    seqs = w.seqs()
    q = dev_u16(np.concatenate(q_list))
    out = t.zeros_like(q)
    size = pkv.window_decode_ws_size(w.lay, seqs, hq, w.window, w.sinks)
    ws = t.full((max(64, size // 4),), float("nan"), dtype=t.float32, device="cuda") if size else None
    pkv.window_decode(w.lay, seqs, 0, hq, w.window, w.sinks, q, out, ws, **new)
    return host_u16(out)


NAN, INF, NINF = 0x7FC1, 0x7F80, 0xFF80
# what KV head 0 of the first stream (or its heads' queries) holds, as (tensor,
# position from the stream's end, dim, bits); each is read by the query
BAD = [[("k", 50, 3, NAN)], [("v", 50, 3, NAN)], [("k", 1, 3, NAN)], [("q", 0, 5, NAN)], [("k", 50, 3, INF)],
       [("q", 0, 5, INF)], [("v", 1, 3, INF), ("v", 50, 3, NINF)], [("k", p, 0, NAN) for p in range(1, 301)]]


@pytest.mark.parametrize("fmt", FMT)
@pytest.mark.parametrize("case", range(len(BAD)))
@pytest.mark.parametrize("window,streams", [(100, 1), (100, 40), (2000, 40), (6000, 2)])
def test_what_is_not_finite_where_it_is_read_is_not_finite_in_the_output(window, streams, case, fmt):
    hq, hkv, sinks, length = 8, 2, 4, 300 if window < 2000 else 6200
    grp = hq // hkv
    lay = pkv.layout(1, hkv, 256, 0, fmt)
    ss = streams_of([length] + [200] * (streams - 1), hkv, seed=61)
    q = queries_of([1] * streams, hq, seed=62)
    clean = Windowed(lay, ss, [1] * streams, window, sinks, 16, seed=5).reference(0, q)
    for what, back, dim, bits in BAD[case]:
        if what == "q":
            q[0][0, :grp, dim] = bits
        else:
            getattr(ss[0], what)[0][length - back, 0, dim] = bits
    w = Windowed(lay, ss, [1] * streams, window, sinks, 16, seed=5)
    got = run(w, hq, q)
    with np.errstate(all="ignore"):
        want = attend(values(ss[0].k[0], fmt), values(ss[0].v[0], fmt), q[0], length, window, sinks)
    odd = (got[0, :grp] & 0x7F80) == 0x7F80
    dims = sorted({d for what, _, d, _ in BAD[case] if what == "v"})
    if dims:                  # of e4m3 rows the other dims share the scale that is not finite
        assert odd[:, dims].all() and (fmt == pkv.KV_E4M3 or odd.sum() == odd[:, dims].sum())
    else:                     # a score of -inf (an infinite key against the query's sign) is a weight of 0
        assert np.array_equal(odd, ~np.isfinite(want[0, :grp])) and odd.any()
    rest = np.concatenate([got[0, grp:].ravel(), got[1:].ravel()])
    ok, report = within_tol(rest, np.concatenate([clean[0, grp:].ravel(), clean[1:].ravel()]))
    assert ok, report


def test_e4m3_rows_whose_scale_is_not_finite():
    # a V scale of inf or NaN set in the cache: not a weight of zero
    t = torch()
    lay = pkv.layout(1, 1, 256, 0, pkv.KV_E4M3)
    s = streams_of([120], 1, seed=8)
    q = queries_of([1], 4)
    for pos in (3, 64, 119):
        for value in (float("inf"), float("nan")):
            w = Windowed(lay, s, [1], 60, 4, 16, seed=2)
            table = next(x for x in w.keep if x.dtype == t.int32).cpu().numpy()[:-1]
            at = pkv.pg_row(lay, w.pgs[0], table, 0, pkv.VS, 0, pos)
            w._body(0).view(t.uint8)[at:at + 4].view(t.float32)[0] = value
            assert ((run(w, 4, q) & 0x7F80) == 0x7F80).all(), (pos, value)


def test_e4m3_queries_beyond_fp16():
    # queries of bf16's range against keys as small or large the other way: the
    # scores, and so the outputs, are those of the definition
    lay = pkv.layout(1, 2, 256, 0, pkv.KV_E4M3)
    for e in (-40, -18, 14, 20, 60):
        ss = streams_of([200, 90], 2, seed=70)
        for s in ss:
            s.k[0] = synth.scale_pow2(s.k[0], -e)
        q = [synth.scale_pow2(x, e) for x in queries_of([2, 1], 8, seed=71)]
        w = Windowed(lay, ss, [2, 1], 64, 4, 16, seed=1)
        ok, report = within_tol(run(w, 8, q), w.reference(0, q))
        assert ok, (e, report)


# calls of more CTAs than the GPU holds that the cost model leaves to clusters, in
# waves: 384 CTAs of 8 pieces, of up to 32 columns in two passes and of 16; a few
# streams with fewer new tokens, and one without
@pytest.mark.parametrize("fmt,top", [(pkv.KV_BF16, 4), (pkv.KV_E4M3, 4), (pkv.KV_E4M3, 2)])
def test_clusters_in_waves(fmt, top):
    t = torch()
    hq, hkv, window, sinks, idx = 16, 2, 4900, 4, 128     # pieces of some 570 keys
    lay = pkv.layout(1, hkv, 256, idx, fmt)
    n_new = [top] * 20 + [1, top, 0, top]
    lens = [int(x) for x in np.linspace(4200, 6300, 22)] + [700, 5000]
    base = streams_of([6300] * 2, hkv, idx, seed=300)          # two streams' rows, each at many lengths
    streams = [synth.Stream(n, base[i & 1].k, base[i & 1].v, base[i & 1].ik) for i, n in enumerate(lens)]
    for s in streams:
        s.k, s.v, s.ik = (x[:, :s.length] for x in (s.k, s.v, s.ik))
    q = queries_of(n_new, hq, seed=301)
    a = Windowed(lay, streams, n_new, window, sinks, 64, seed=1, fused=True)
    b = Windowed(lay, streams, n_new, window, sinks, 64, seed=1, fused=True)
    pkv.store(lay, b.seqs(), 0, *b.new_rows(0))
    k, v, ik = a.new_rows(0)
    got = run(a, hq, q, k_new=k, v_new=v, ik_new=ik)
    assert np.array_equal(got, run(b, hq, q))
    assert t.equal(a.bufs[0], b.bufs[0])
    rows = np.split(got, np.cumsum(n_new)[:-1])
    for i in (0, 7, 20, 21, 23):
        w = Windowed(lay, streams[i:i + 1], n_new[i:i + 1], window, sinks, 256, seed=i)
        ok, report = within_tol(rows[i], w.reference(0, q[i:i + 1]))
        assert ok, (i, report)
        assert np.array_equal(run(w, hq, q[i:i + 1]), rows[i])      # alone: one cluster a KV head, or two
    for _ in range(10):
        assert np.array_equal(run(b, hq, q), got)
