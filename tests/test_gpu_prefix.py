"""Decode over shared pages on the GPU: against the definition in float64, over page sizes, formats, groups and masks."""
import numpy as np
import pytest

from paged_kv_cache_pg_gb300 import pkv

from gpu_setup import torch
from prefix_setup import Shared
from rope_setup import bf16_bits, bf16_values

pytestmark = pytest.mark.gpu

BF, E4 = pkv.KV_BF16, pkv.KV_E4M3

# a small call's streams are decoded each by itself, and together beside a large group
TOGETHER = pytest.mark.parametrize("ballast", [0, 24], ids=["alone", "together"])


@pytest.fixture(scope="module", autouse=True)
def built():
    from paged_kv_cache_pg_gb300 import build
    build.build()
    pkv.load()


@TOGETHER
@pytest.mark.parametrize("fmt", [BF, E4])
@pytest.mark.parametrize("ptok,pages", [(128, 1), (256, 3), (16, 5), (48, 9), (64, 4), (4, 1), (4, 67), (20, 20)])
def test_two_streams(fmt, ptok, pages, ballast):
    lay = pkv.layout(2, 2, 256, 128, fmt)
    s = Shared(lay, [([3, 40], pages)], 1, ptok, layer=1, ballast=ballast)
    s.check(s.call())


@TOGETHER
@pytest.mark.parametrize("fmt", [BF, E4])
@pytest.mark.parametrize("ptok", [16, 20, 128])
@pytest.mark.parametrize("hkv,hq,new", [(1, 4, 1), (2, 16, 2), (1, 32, 1), (3, 3, 4), (4, 20, 3)])
def test_groups_of_every_kind(fmt, ptok, hkv, hq, new, ballast):
    """Groups that share, one stream alone, one that shares nothing, streams without queries."""
    lay = pkv.layout(1, hkv, 256, 0, fmt)
    groups = [([new, 70, 33], 700 // ptok), ([90], 5), ([21, 300], 0), ([15, 16, 17, 18, 500], 1300 // ptok), ([64, 9], 2)]
    n_new = [new, new, 0, new, new, new, 0, new, new, 0, new, new, 0]
    s = Shared(lay, groups, n_new, ptok, fused=True, n_q_heads=hq, seed=hq, ballast=ballast)
    s.check(s.call())


@TOGETHER
@pytest.mark.parametrize("fmt,ptok", [(BF, 256), (BF, 48), (E4, 128), (E4, 4)])
def test_long_prefix(fmt, ptok, ballast):
    """Eight samples of one prompt of 9,000 positions: splits over the whole GPU."""
    lay = pkv.layout(1, 2, 256, 128, fmt)
    s = Shared(lay, [([400, 5, 1, 77, 128, 129, 250, 31], 9000 // ptok)], 1, ptok, n_q_heads=16, ballast=ballast)
    s.check(s.call())


@pytest.mark.parametrize("fmt", [BF, E4])
def test_many_rows(fmt):
    """64 streams of 8 columns: two M-tiles of 256 rows a KV head; then draft windows: 40 x 32 columns, five."""
    lay = pkv.layout(1, 2, 256, 0, fmt)
    for pages in (9, 32):
        s = Shared(lay, [([1 + i for i in range(64)], pages)], 1, 128, n_q_heads=16)
        s.check(s.call())
    s = Shared(lay, [([4 + i for i in range(40)], 30)], 4, 64, n_q_heads=16, fused=True)
    s.check(s.call())


@pytest.mark.parametrize("ballast", [0, 20], ids=["alone", "together"])
@pytest.mark.parametrize("rows_streams,new,hq", [(2, 1, 1), (33, 1, 1), (43, 3, 1), (2, 4, 8), (9, 1, 29)])
def test_row_counts(rows_streams, new, hq, ballast):
    """M-tiles of 2 to 261 rows: halves of a pair that are empty, odd, full."""
    lay = pkv.layout(1, 1, 256, 0)
    s = Shared(lay, [([new + 2 * i for i in range(rows_streams)], 3)], new, 64, n_q_heads=hq, seed=rows_streams, ballast=ballast)
    s.check(s.call())


@pytest.mark.parametrize("fmt", [BF, E4])
def test_largest(fmt):
    """All streams with all the columns a call takes: eight units of 256 rows; and 64 KV heads."""
    s = Shared(pkv.layout(1, 2, 256, 0, fmt), [([4 + 3 * i for i in range(64)], 8)], 4, 128, n_q_heads=16, fused=True)
    s.check(s.call())
    s = Shared(pkv.layout(1, 64, 256, 0, fmt), [([5, 20, 33], 2)], 2, 64, n_q_heads=64, fused=True, ballast=24)
    s.check(s.call())


@TOGETHER
@pytest.mark.parametrize("fmt", [BF, E4])
@pytest.mark.parametrize("gain", [8.0, 16.0, 64.0])
def test_peaked(fmt, gain, ballast):
    """A softmax on few keys, whose maximum grows from tile to tile; one far above near the prefix's end."""
    lay = pkv.layout(1, 2, 256, 0, fmt)
    s = Shared(lay, [([40, 60, 7], 12)], 2, 128, n_q_heads=8, gain=gain, seed=3, ballast=ballast)
    s.check(s.call())
    if gain == 8.0:
        s = Shared(lay, [([40, 60, 7], 12)], 1, 128, n_q_heads=2, gain=gain, late=True, seed=4, ballast=ballast)
        s.check(s.call())


@TOGETHER
@pytest.mark.parametrize("spread", [4, 12])
def test_value_rows_of_many_sizes(spread, ballast):
    """bf16 rows within fp16's normal range; e4m3 rows over 2^+-20 and 2^+-38."""
    s = Shared(pkv.layout(1, 2, 256, 0), [([9, 4], 6)], 1, 128, spread=spread, ballast=ballast)
    s.check(s.call()) if spread == 4 else None
    s = Shared(pkv.layout(1, 2, 256, 0, E4), [([9, 4], 6)], 1, 128, spread=20 if spread == 4 else 38, ballast=ballast)
    s.check(s.call())
    s = Shared(pkv.layout(1, 2, 256, 0, E4), [([9, 4], 6)], 1, 128, spread=20, gain=16.0, ballast=ballast)
    s.check(s.call())


@TOGETHER
def test_zero_rows_e4m3(ballast):
    """Value rows of zeros (scale 0) that take all the weight, and whole tiles of them."""
    lay = pkv.layout(1, 1, 256, 0, E4)
    s = Shared(lay, [([9, 4], 4)], 1, 128, n_q_heads=4, gain=8.0, ballast=ballast)
    t, keep = torch(), s.v[0][:512].copy()
    keep[:256] = 0
    for i in range(2):
        s.v[i][:512] = keep
        pkv.store(lay, [pkv.seq(s.pgs[i], 512, 512)], 0, s.dev(s.k[i][:512]), s.dev(s.v[i][:512]))
    t.cuda.synchronize()
    s.check(s.call())


@TOGETHER
@pytest.mark.parametrize("fmt", [BF, E4])
@pytest.mark.parametrize("ptok", [16, 20, 128])
def test_stores_as_store_does(fmt, ptok, ballast):
    lay = pkv.layout(2, 2, 256, 128, fmt)
    groups = [([3, 40, 17], 8), ([33, 5], 0)]
    a = Shared(lay, groups, [1, 2, 3, 1, 4], ptok, fused=True, n_q_heads=16, layer=1, ballast=ballast)
    b = Shared(lay, groups, [1, 2, 3, 1, 4], ptok, fused=True, n_q_heads=16, layer=1, ballast=ballast)
    pkv.store(lay, b.seqs, 1, b.k_new, b.v_new, b.ik_new)
    b.fused = False
    before, one, two = b.mem.clone(), a.call(), b.call()
    assert torch().equal(a.mem, b.mem) and torch().equal(b.mem, before) and torch().equal(one, two)
    a.check(one)


@TOGETHER
@pytest.mark.parametrize("fmt", [BF, E4])
def test_bits_do_not_follow_the_pages(fmt, ballast):
    """The same call over other page ids, and twice: the same bits."""
    lay = pkv.layout(1, 2, 256, 128, fmt)
    a = Shared(lay, [([30, 7, 200], 20)], 1, 48, n_q_heads=16, seed=1, ballast=ballast)
    one = a.call()
    perm = np.random.default_rng(9).permutation(a.n_pages)
    t = torch()
    mem = t.empty_like(a.mem)
    mem[t.from_numpy(perm).cuda()] = a.mem
    tables = [t.from_numpy(perm[x].astype(np.int32)).cuda() for x in a.tables]
    seqs = [pkv.seq(pkv.pg(mem, x, a.ps, 48, a.n_pages), n, m) for x, n, m in zip(tables, a.lens, a.new)]
    two = t.full_like(one, 77)
    pkv.prefix_decode(lay, seqs, a.groups, 0, 16, a.dq, two, a.ws())
    assert t.equal(one, two) and t.equal(one, a.call())


@TOGETHER
def test_as_decode_of_the_streams_alone(ballast):
    """Sharing changes roundings only: against pkv_decode of the same streams, within two bounds."""
    lay = pkv.layout(1, 2, 256, 0)
    s = Shared(lay, [([30, 70], 9), ([200, 4], 3)], 1, 64, n_q_heads=16, ballast=ballast)
    got, t = s.call(), torch()
    ws = t.empty(max(64, pkv.decode_ws_size(lay, s.seqs, 16) // 4), device="cuda")
    alone = t.full_like(got, 77)
    pkv.decode(lay, s.seqs, 0, 16, s.dq, alone, ws)
    s.check(got)
    s.check(alone)


@pytest.mark.parametrize("fmt", [BF, E4])
@pytest.mark.parametrize("hkv,hq,new", [(1, 4, 1), (2, 16, 2), (4, 20, 3)])
def test_together_or_alone(fmt, hkv, hq, new):
    """Few shared rows: the bits of pkv_window_decode of the same streams; many: others."""
    t, lay = torch(), pkv.layout(1, hkv, 256, 0, fmt)
    for ballast in (0, 24):
        s = Shared(lay, [([30, 70, 200], 9)], new, 64, n_q_heads=hq, ballast=ballast)
        got, n = s.call(), max(s.lens)
        ws = t.empty(max(64, pkv.window_decode_ws_size(lay, s.seqs, hq, n, 0) // 4), device="cuda")
        alone = t.full_like(got, 77)
        pkv.window_decode(lay, s.seqs, 0, hq, n, 0, s.dq, alone, ws)
        assert t.equal(got, alone) == (ballast == 0)
        s.check(got)


def test_nothing_shared():
    """No groups at all are no groups of no streams; groups without shared pages; single streams: no workspace of partials needed."""
    lay = pkv.layout(1, 2, 256, 0)
    s = Shared(lay, [([30, 70], 0), ([200], 0)], 1, 64, n_q_heads=8)
    s.check(s.call())
    s = Shared(lay, [([30], 4), ([200], 2)], 1, 64, n_q_heads=8)
    assert pkv.prefix_decode_ws_size(lay, s.seqs, s.groups, 8) == 0
    s.check(s.call(ws=torch().empty(64, device="cuda")))


@TOGETHER
@pytest.mark.parametrize("fmt", [BF, E4])
def test_one_workspace_for_all_lengths(fmt, ballast):
    """The size for the longest own parts covers shorter ones, whatever is shared; nothing behind it is written."""
    t = torch()
    lay = pkv.layout(1, 2, 256, 0, fmt)
    big = Shared(lay, [([700, 700, 700], 0)], 4, 64, n_q_heads=16, ballast=ballast)
    size = pkv.prefix_decode_ws_size(lay, big.seqs, big.groups, 16) // 4
    for own, pages, new in (([700, 3, 650], 40, 3), ([1, 1, 1], 90, 1), ([640, 641, 4], 1, 4), ([100, 90, 80], 7, 2)):
        s = Shared(lay, [(own, pages)], [min(new, n) for n in own], 64, n_q_heads=16, ballast=ballast)
        assert pkv.prefix_decode_ws_size(lay, s.seqs, s.groups, 16) <= 4 * size
        ws = t.full((size + 64,), 3.0, device="cuda")
        s.check(s.call(ws=ws[:size]))
        assert (ws[size:] == 3.0).all()


@TOGETHER
@pytest.mark.parametrize("where", ["k", "v"])
@pytest.mark.parametrize("fmt", [BF, E4])
def test_not_finite(fmt, where, ballast):
    """A NaN or an infinity in a shared row comes out as not finite, for every query that reads it; others stay."""
    lay = pkv.layout(1, 2, 256, 0, fmt)
    s = Shared(lay, [([9, 4], 3), ([5, 7], 2)], 1, 64, n_q_heads=4, ballast=ballast)
    rows = getattr(s, where)
    for i in range(2):
        rows[i][100, 1, 5] = 0x7FC0 if where == "k" else 0x7F80
        pkv.store(lay, [pkv.seq(s.pgs[i], 192, 192)], 0, s.dev(s.k[i][:192]), s.dev(s.v[i][:192]))
    st = torch().zeros(1, dtype=torch().int32, device="cuda")
    got = bf16_values(s.call(status=st).cpu().numpy().view(np.uint16))[:-1]
    bad = ~np.isfinite(got)
    assert bad[:2, 2:].any(-1).all() and not bad[:2, :2].any() and not bad[2:].any()
    assert int(st) & ~pkv.DEV_RANGE == 0


@TOGETHER
@pytest.mark.parametrize("fmt", [BF, E4])
@pytest.mark.parametrize("ptok", [64, 20])
@pytest.mark.parametrize("where,dim", [("k", 5), ("v", 5), ("v", 200)])
def test_not_finite_in_an_own_row(fmt, ptok, where, dim, ballast):
    """A stream's own row that is not finite: its outputs of that KV head are not, and no other stream's change by a bit."""
    lay = pkv.layout(1, 2, 256, 0, fmt)
    s = Shared(lay, [([90, 40, 33], 3), ([50, 60], 2)], [1, 2, 1, 1, 3], ptok, n_q_heads=4, ballast=ballast)
    good = bf16_values(s.call().cpu().numpy().view(np.uint16))[:-1]
    n = s.lens[1]
    getattr(s, where)[1][n - 15, 0, dim] = 0x7FC0
    pkv.store(lay, [pkv.seq(s.pgs[1], n, n)], 0, s.dev(s.k[1]), s.dev(s.v[1]))
    st = torch().zeros(1, dtype=torch().int32, device="cuda")
    got = bf16_values(s.call(status=st).cpu().numpy().view(np.uint16))[:-1]
    assert np.isnan(got[1:3, :2]).any(-1).all() and int(st) & ~pkv.DEV_RANGE == 0
    rest = np.ones(got.shape, bool)
    rest[1:3, :2] = False
    assert np.array_equal(got[rest], good[rest])


@TOGETHER
@pytest.mark.parametrize("ptok", [64, 20])
@pytest.mark.parametrize("bits", [0x7F80, 0x7FC0, 0xFF80])
def test_not_finite_scale_of_an_own_row(ptok, bits, ballast):
    """... of an e4m3 value row: its stream's outputs of that KV head are not finite, no other's change by a bit."""
    lay = pkv.layout(1, 2, 256, 0, E4)
    s = Shared(lay, [([90, 40, 33], 3), ([50, 60], 2)], [1, 2, 1, 1, 3], ptok, n_q_heads=4, ballast=ballast)
    good = s.call()
    at = pkv.pg_row(lay, s.pgs[1], s.tables[1], 0, pkv.VS, 1, s.lens[1] - 15)
    s.mem.view(-1)[at // 2:at // 2 + 2] = s.dev(np.array([0, bits], np.uint16))   # (e4m3 offsets are in bytes)
    st = torch().zeros(1, dtype=torch().int32, device="cuda")
    got = s.call(status=st)
    a, b = (bf16_values(x.cpu().numpy().view(np.uint16))[:-1] for x in (got, good))
    assert (~np.isfinite(a[1:3, 2:])).any(-1).all() and int(st) & ~pkv.DEV_RANGE == 0
    rest = np.ones(a.shape, bool)
    rest[1:3, 2:] = False
    assert np.array_equal(a[rest], b[rest])


@TOGETHER
def test_values_beyond_fp16_are_reported(ballast):
    """... where shared rows are read together: a stream alone is exact over bf16's range."""
    lay = pkv.layout(1, 1, 256, 0)
    t = torch()
    for top, told in ((65280.0, 0), (70000.0, pkv.DEV_RANGE if ballast else 0)):
        s = Shared(lay, [([9, 4], 3)], 1, 64, n_q_heads=4, ballast=ballast)
        for i in range(2):
            s.v[i][100, 0, 5] = bf16_bits(np.array([top]))[0]
            pkv.store(lay, [pkv.seq(s.pgs[i], 192, 192)], 0, s.dev(s.k[i][:192]), s.dev(s.v[i][:192]))
        st = t.zeros(1, dtype=t.int32, device="cuda")
        out = s.call(status=st)
        assert int(st) == told
        if not told:
            s.check(out)


@TOGETHER
@pytest.mark.parametrize("fmt", [BF, E4])
@pytest.mark.parametrize("ptok", [64, 128, 20])
def test_a_bad_page_is_reported(fmt, ptok, ballast):
    """A shared page id outside the arena: reported, read as page 0, the other group as ever."""
    lay = pkv.layout(1, 1, 256, 0, fmt)
    t = torch()
    s = Shared(lay, [([9, 4], 3), ([5, 7], 6)], 1, ptok, n_q_heads=4, ballast=ballast)
    good = s.call()
    s.mem[0] = 0
    for i in (0, 1):
        s.dev_tables[i][1] = s.n_pages if i else -5
    s.mem.copy_(s.mem)
    st = t.zeros(1, dtype=t.int32, device="cuda")
    out = s.call(status=st)
    assert int(st) & pkv.DEV_BAD_PAGE
    keep = 0 not in s.tables[2] and 0 not in s.tables[3]
    assert not keep or t.equal(out[2:4], good[2:4])


def test_pages_past_4_gb():
    """Shared pages whose byte offsets pass 32 bits."""
    t = torch()
    for fmt in (BF, E4):
        lay = pkv.layout(13, 2, 256, 128, fmt)
        ptok = 256
        ps = pkv.page_elems(lay, ptok)
        n_pages = (5 << 30) // (2 * ps) + 4
        s = Shared(pkv.layout(1, 2, 256, 128, fmt), [([20, 9] * 16, 16)], 1, ptok, n_q_heads=16)
        mem = t.zeros((n_pages, ps), dtype=t.int16, device="cuda")
        ids = np.arange(n_pages - 1, n_pages - 17, -1)
        tabs = [t.from_numpy(np.append(ids, n_pages - 17 - i if i else 0).astype(np.int32)).cuda() for i in range(32)]
        pgs = [pkv.pg(mem, x, ps, ptok, n_pages) for x in tabs]
        for i in range(32):
            n = s.lens[i]
            pkv.store(lay, [pkv.seq(pgs[i], n, n)], 12, s.dev(s.k[i]), s.dev(s.v[i]), t.zeros((n, 128), dtype=t.int16, device="cuda"))
        seqs = [pkv.seq(g, n, 1) for g, n in zip(pgs, s.lens)]
        out, st = t.full((33, 16, 256), 77, dtype=t.int16, device="cuda"), t.zeros(1, dtype=t.int32, device="cuda")
        pkv.prefix_decode(lay, seqs, [(32, 16)], 12, 16, s.dq, out, s.ws(), status=st)
        assert int(st) == 0
        s.check(out)
        del mem


@TOGETHER
def test_a_graph_and_calls_in_a_row(ballast):
    """Captured on a stream of its own and replayed on new queries; calls of two workspaces in a row on another."""
    t = torch()
    lay = pkv.layout(1, 2, 256, 128)
    a = Shared(lay, [([30, 7, 200], 20)], 1, 64, fused=True, n_q_heads=16, seed=1, ballast=ballast)
    b = Shared(lay, [([3, 70], 9)], 1, 64, fused=True, n_q_heads=16, seed=2, ballast=ballast)
    ws, wsb = a.ws(), b.ws()
    out, outb = (t.full((n + ballast, 16, 256), 77, dtype=t.int16, device="cuda") for n in (4, 3))
    st = t.zeros(1, dtype=t.int32, device="cuda")
    side, other = t.cuda.Stream(), t.cuda.Stream()
    t.cuda.synchronize()
    with t.cuda.stream(side):
        a.call(ws=ws, out=out, status=st)
        side.synchronize()
        g = t.cuda.CUDAGraph()
        with t.cuda.graph(g, stream=side):
            a.call(ws=ws, out=out, status=st)
    for seed in range(3):
        a.q = bf16_bits(np.random.default_rng(seed).standard_normal(a.q.shape))
        with t.cuda.stream(side):
            a.dq[:3].copy_(a.dev(a.q))
            g.replay()
        with t.cuda.stream(other):
            for _ in range(3):
                b.call(ws=wsb, out=outb, status=st)
        t.cuda.synchronize()
        a.check(out)
        b.check(outb)
    assert int(st) == 0


@TOGETHER
@pytest.mark.parametrize("fmt", [BF, E4])
@pytest.mark.parametrize("other", [20, 48, 128])
def test_arenas_of_their_own(fmt, other, ballast):
    """Groups of two arenas with pages of their own size, and a contiguous stream between them, in one call."""
    t, lay, hq = torch(), pkv.layout(1, 2, 256, 0, fmt), 8
    a = Shared(lay, [([9, 70], 7)], [1, 2], other, n_q_heads=hq, seed=1)
    c = Shared(lay, [([333], 0)], 3, 64, n_q_heads=hq, seed=2)
    b = Shared(lay, [([33, 4, 150], 5), ([20, 21], 1)], 2, 64, n_q_heads=hq, seed=3, ballast=ballast)
    flat = t.full((1, pkv.page_elems(lay, 336)), 0x7FC1, dtype=t.int16, device="cuda")
    alone = pkv.Pg(flat.data_ptr(), None, flat.shape[1], 336, 1, 1, 0)
    pkv.store(lay, [pkv.seq(alone, 333, 333)], 0, c.dev(c.k[0]), c.dev(c.v[0]))
    seqs, groups = a.seqs + [pkv.seq(alone, 333, 3)] + b.seqs, a.groups + [(1, 0)] + b.groups
    q, st = t.cat([a.dq, c.dq, b.dq]), t.zeros(1, dtype=t.int32, device="cuda")
    ws = t.full((max(64, pkv.prefix_decode_ws_size(lay, seqs, groups, hq) // 4),), float("nan"), device="cuda")
    out = t.full((q.shape[0] + 1, hq, 256), 77, dtype=t.int16, device="cuda")
    pkv.prefix_decode(lay, seqs, groups, 0, hq, q, out, ws, status=st)
    assert int(st) == 0
    end, at = out[-1:], 0
    for s in (a, c, b):
        n = s.dq.shape[0]
        s.check(t.cat([out[at:at + n], end]))
        at += n


@TOGETHER
@pytest.mark.parametrize("fmt", [BF, E4])
def test_storing_calls_in_a_row(fmt, ballast):
    """Thirty tokens of each stream, stored by the calls, one call behind another: the bits of calls whose rows were there before."""
    t, lay, hq, steps = torch(), pkv.layout(1, 2, 256, 128, fmt), 16, 30
    s = Shared(lay, [([60, 90, 75], 9), ([40], 0)], 1, 64, n_q_heads=hq, ballast=ballast)
    mem, nan = s.mem.clone(), t.full((4 * steps, 2, 256), 0x7FC1, dtype=t.int16, device="cuda")
    pgs = [pkv.pg(mem, x, s.ps, 64, s.n_pages) for x in s.dev_tables]
    pkv.store(lay, [pkv.seq(g, n, steps) for g, n in zip(pgs[:4], s.lens)], 0, nan, nan, nan[:, 0, :128].contiguous())
    ik, ws = t.zeros((4 + ballast, 128), dtype=t.int16, device="cuda"), s.ws()
    st = t.zeros(1, dtype=t.int32, device="cuda")
    calls = []
    for step in range(steps):
        lens = [n - steps + 1 + step if i < 4 else n for i, n in enumerate(s.lens)]
        new = [t.cat([s.dev(np.stack([x[i][lens[i] - 1] for i in range(4)])), y[4:]]) for x, y in ((s.k, s.k_new), (s.v, s.v_new))]
        calls.append((lens, new, t.full_like(s.dq, 77), t.full_like(s.dq, 77)))
    t.cuda.synchronize()
    for lens, (k, v), out, _ in calls:
        pkv.prefix_decode(lay, [pkv.seq(g, n, 1) for g, n in zip(pgs, lens)], s.groups, 0, hq, s.dq, out, ws, status=st, k_new=k, v_new=v, ik_new=ik)
    for lens, _, _, out in calls:
        pkv.prefix_decode(lay, [pkv.seq(g, n, 1) for g, n in zip(s.pgs, lens)], s.groups, 0, hq, s.dq, out, ws, status=st)
    assert int(st) == 0 and all(t.equal(a, b) for _, _, a, b in calls)


@pytest.mark.parametrize("forks,n", [(5, 1000), (47, 4000)])
def test_forks_decoding_token_by_token(forks, n):
    """As it is used: a prompt stored and forked, its page copied, then steps of rope_store and prefix_decode of all forks, against
    decode over the same cache."""
    t = torch()
    rng = np.random.default_rng(12)
    lay, hq, ptok, pages = pkv.layout(1, 2, 256, 128), 16, 64, 80 if forks == 5 else 300
    ps = pkv.page_elems(lay, ptok)
    mem = t.full((pages, ps), 0x7FC1, dtype=t.int16, device="cuda")
    arena = pkv.Arena(lay, ptok, mem)
    rows = lambda *shape: Shared.dev(bf16_bits(rng.standard_normal(shape)))  # noqa: E731
    rope = pkv.rope(64, 1e6)
    prompt = arena.take(-(-n // ptok))
    table = t.from_numpy(prompt).cuda()
    pkv.rope_store(lay, [pkv.seq(arena.pg(table), n, n)], 0, rope, rows(n, 2, 256), rows(n, 2, 256), rows(n, 128))
    streams = [prompt]
    for _ in range(forks):
        ids, copy = arena.fork(prompt, n)
        pkv.pages_copy(lay, ptok, mem, pages, [copy[0]], [copy[1]], [copy[2]])
        streams.append(ids)
    tables = [t.from_numpy(np.concatenate([x, arena.take(2)]).astype(np.int32)).cuda() for x in streams]
    groups, m = pkv.groups([(forks + 1, n // ptok)]), forks + 1
    st = t.zeros(1, dtype=t.int32, device="cuda")
    q, out, alone = (t.empty((m, hq, 256), dtype=t.int16, device="cuda") for _ in range(3))
    last = [pkv.seq(arena.pg(x), n + 100, 1) for x in tables]
    ws = t.empty(pkv.prefix_decode_ws_size(lay, last, groups, hq) // 4, device="cuda")
    ws2 = t.empty(max(64, pkv.decode_ws_size(lay, last, hq) // 4), device="cuda")
    for step in range(70):
        seqs = [pkv.seq(arena.pg(x), n + 1 + step, 1) for x in tables]
        pkv.rope_store(lay, seqs, 0, rope, rows(m, 2, 256), rows(m, 2, 256), rows(m, 128), n_q_heads=hq, q=rows(m, hq, 256), q_out=q, status=st)
        pkv.prefix_decode(lay, seqs, groups, 0, hq, q, out, ws, status=st)
        pkv.decode(lay, seqs, 0, hq, q, alone, ws2, status=st)
        if step % 23 == 0:
            x, y = (bf16_values(z.cpu().numpy().view(np.uint16)) for z in (out, alone))
            # both within 2^-11 of a value of at most 5, and rounded
            assert (np.abs(x - y) <= 2 * 2.0 ** -8 * np.maximum(np.abs(x), np.abs(y)) + 2 * 2.0 ** -11 * 5).all()
    assert int(st) == 0
