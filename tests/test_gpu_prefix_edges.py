"""Decode over shared pages on the GPU: units of odd shapes, rows that some tokens must not see, workspaces, routes."""
import numpy as np
import pytest

from paged_kv_cache_pg_gb300 import pkv

from gpu_setup import torch
from prefix_setup import Shared
from rope_setup import bf16_bits, bf16_values

pytestmark = pytest.mark.gpu

BF, E4 = pkv.KV_BF16, pkv.KV_E4M3


@pytest.fixture(scope="module", autouse=True)
def built():
    from paged_kv_cache_pg_gb300 import build
    build.build()
    pkv.load()


def decoded_alone(s, out):
    """Whether these are the bits of pkv_window_decode over all positions, each stream by itself (its rows are stored by now)."""
    t, n = torch(), max(s.lens)
    ws = t.empty(max(64, pkv.window_decode_ws_size(s.lay, s.seqs, s.n_q_heads, n, 0) // 4), device="cuda")
    alone = t.full_like(out, 77)
    pkv.window_decode(s.lay, s.seqs, s.layer, s.n_q_heads, n, 0, s.dq, alone, ws)
    return t.equal(out, alone)


@pytest.mark.parametrize("fmt", [BF, E4])
@pytest.mark.parametrize("ptok", [64, 20])
@pytest.mark.parametrize("own", [1, 130, 700])
def test_units_of_one_row(fmt, ptok, own):
    """A stream of one query head a KV head that shares nothing, beside groups that do: the second CTA of its pair has no row.
    Splits of one tile and of several, calls in a row."""
    lay = pkv.layout(1, 1, 256, 0, fmt)
    s = Shared(lay, [([own], 0), ([3, 40], 700 // ptok), ([own], 2)], 1, ptok, n_q_heads=1, seed=own, ballast=24)
    ws = s.ws()
    outs = [s.call(ws=ws) for _ in range(4)]
    s.check(outs[0])
    assert not decoded_alone(s, outs[0])
    assert all(torch().equal(outs[0], x) for x in outs[1:])


@pytest.mark.parametrize("fmt", [BF, E4])
@pytest.mark.parametrize("ptok", [128, 20])
def test_a_unit_of_256_rows_and_one_of_one(fmt, ptok):
    """63 streams of four columns and one of five: the second unit is one row, whose stream's other rows are the first unit's."""
    lay = pkv.layout(1, 1, 256, 0, fmt)
    s = Shared(lay, [([5 + i for i in range(64)], 4096 // ptok)], [4] * 63 + [5], ptok, n_q_heads=1, fused=True)
    out = s.call()
    s.check(out)
    assert not decoded_alone(s, out)


@pytest.mark.parametrize("fmt", [BF, E4])
@pytest.mark.parametrize("hkv,hq,new,pages", [(40, 40, 1, 11), (8, 16, 2, 190), (2, 16, 1, 830)])
def test_the_told_workspace_covers_one_stream_left(fmt, hkv, hq, new, pages):
    """Streams of a group end one after another; the size told while all decode, over less, is enough for the last one alone."""
    t, lay, ptok = torch(), pkv.layout(1, hkv, 256, 0, fmt), 64
    first = Shared(lay, [([20, 9], 1), ([30], 0)], new, ptok, n_q_heads=hq)
    size = pkv.prefix_decode_ws_size(lay, first.seqs, first.groups, hq) // 4
    for live in ([new, new, new], [0, new, 0], [new, 0, new], [1, 0, 0]):
        s = Shared(lay, [([20, 9], pages), ([30], 0)], live, ptok, n_q_heads=hq)
        assert pkv.prefix_decode_ws_size(lay, s.seqs, s.groups, hq) <= 4 * size
        ws = t.full((size + 64,), 3.0, device="cuda")
        s.check(s.call(ws=ws[:size]))
        assert (ws[size:] == 3.0).all()


@pytest.mark.parametrize("fmt", [BF, E4])
@pytest.mark.parametrize("ptok", [64, 20])
@pytest.mark.parametrize("where,value", [("k", np.nan), ("v", np.nan), ("v", np.inf), ("v", 70000.0)])
@pytest.mark.parametrize("back", [1, 2, 3])
def test_a_draft_token_does_not_read_later_rows_that_are_not_finite(fmt, ptok, where, value, back):
    """The row `back` before the end of a stream of four draft tokens: those before it keep their bits, as all other streams."""
    t, lay = torch(), pkv.layout(1, 2, 256, 0, fmt)
    s = Shared(lay, [([90, 40, 33], 3), ([20], 0)], [1, 4, 4, 2], ptok, n_q_heads=4, ballast=24)
    good = s.call()
    assert not decoded_alone(s, good)
    n = s.lens[1]
    getattr(s, where)[1][n - back, 0, [5, 200]] = bf16_bits(np.array([value]))[0]
    pkv.store(lay, [pkv.seq(s.pgs[1], n, n)], 0, s.dev(s.k[1]), s.dev(s.v[1]))
    st = t.zeros(1, dtype=t.int32, device="cuda")
    out = s.call(status=st)
    a, b = (bf16_values(x.cpu().numpy().view(np.uint16))[:-1] for x in (out, good))
    if fmt == E4 and value == 70000.0:
        # A row of 70,000 is finite there: codes of up to 448 with a scale of 70000 / 448.  The reference that a tile's
        # weights are rounded against follows its scales, so others' bits may change: all of it against the definition.
        assert int(st) == 0
        s.check(out)
        return
    reads = np.zeros(a.shape, bool)
    reads[5 - back:5, :2] = True      # tokens 1 .. 4 are the stream's
    assert np.array_equal(a[~reads], b[~reads])
    assert (~np.isfinite(a[5 - back:5, :2])).any(-1).all() and int(st) & ~pkv.DEV_RANGE == 0
    assert where == "k" or int(st) == pkv.DEV_RANGE


@pytest.mark.parametrize("ptok", [64, 20])
@pytest.mark.parametrize("bits", [0x7F80, 0x7FC0])
def test_nor_later_scales_that_are_not_finite(ptok, bits):
    """... of an e4m3 value row."""
    lay = pkv.layout(1, 2, 256, 0, E4)
    s = Shared(lay, [([90, 40, 33], 3)], [1, 4, 4], ptok, n_q_heads=4, ballast=24)
    good = s.call()
    at = pkv.pg_row(lay, s.pgs[1], s.tables[1], 0, pkv.VS, 1, s.lens[1] - 2)
    s.mem.view(-1)[at // 2:at // 2 + 2] = s.dev(np.array([0, bits], np.uint16))   # (e4m3 offsets are in bytes)
    st = torch().zeros(1, dtype=torch().int32, device="cuda")
    a, b = (bf16_values(x.cpu().numpy().view(np.uint16))[:-1] for x in (s.call(status=st), good))
    reads = np.zeros(a.shape, bool)
    reads[3:5, 2:] = True
    assert np.array_equal(a[~reads], b[~reads]) and (~np.isfinite(a[3:5, 2:])).any(-1).all() and int(st) == pkv.DEV_RANGE


SMALL = [([9, 4], 3), ([5, 7], 2)]
ODD = [([90, 40, 33], 3), ([50, 60], 2)]
SHAPES = [   # layers, KV heads, indexer dims, groups, new tokens, page size, query heads, small calls' ballast
    *((2, 2, 128, [([3, 40], pages)], 1, ptok, 8, 24) for ptok, pages in ((128, 1), (256, 3), (16, 5), (48, 9), (64, 4), (4, 1), (4, 67), (20, 20))),
    *((1, hkv, 0, [([new, 70, 33], 700 // ptok), ([90], 5), ([21, 300], 0), ([15, 16, 17, 18, 500], 1300 // ptok), ([64, 9], 2)],
       [new, new, 0, new, new, new, 0, new, new, 0, new, new, 0], ptok, hq, 24)
      for ptok in (16, 20, 128) for hkv, hq, new in ((1, 4, 1), (2, 16, 2), (1, 32, 1), (3, 3, 4), (4, 20, 3))),
    *((1, 1, 0, [([new + 2 * i for i in range(n)], 3)], new, 64, hq, 20) for n, new, hq in ((2, 1, 1), (33, 1, 1), (43, 3, 1), (2, 4, 8), (9, 1, 29))),
    *((1, 2, 128, [([400, 5, 1, 77, 128, 129, 250, 31], 9000 // ptok)], 1, ptok, 16, 24) for ptok in (256, 48, 128, 4)),
    *((1, 2, 0, [([40, 60, 7], 12)], new, 128, hq, 24) for new, hq in ((2, 8), (1, 2))),
    (1, 2, 0, [([9, 4], 6)], 1, 128, 8, 24), (1, 1, 0, [([9, 4], 4)], 1, 128, 4, 24), (1, 1, 0, [([9, 4], 3)], 1, 64, 4, 24),
    *((2, 2, 128, [([3, 40, 17], 8), ([33, 5], 0)], [1, 2, 3, 1, 4], ptok, 16, 24) for ptok in (16, 20, 128)),
    *((1, 2, idx, [([30, 7, 200], 20)], 1, ptok, 16, 24) for idx, ptok in ((128, 48), (128, 64))),
    *((1, 2, 0, [(own, pages)], new, 64, 16, 24) for own, pages, new in (([700, 3, 650], 40, 3), ([1, 1, 1], 90, 1), ([640, 641, 4], 1, 4), ([100, 90, 80], 7, 2))),
    *((1, 2, 0, groups, new, ptok, 4, 24) for groups, new, ptok in ((SMALL, 1, 64), (ODD, [1, 2, 1, 1, 3], 64), (ODD, [1, 2, 1, 1, 3], 20))),
    *((1, 1, 0, [([9, 4], 3), ([5, 7], 6)], 1, ptok, 4, 24) for ptok in (64, 128, 20)),
    (1, 2, 128, [([60, 90, 75], 9), ([40], 0)], 1, 64, 16, 24),
]


@pytest.mark.parametrize("fmt", [BF, E4])
@pytest.mark.parametrize("shape", range(len(SHAPES)))
def test_calls_meant_to_read_together_do(fmt, shape):
    """The shapes that stand for calls whose streams are read together, beside a large group, are: not the windowed decode's bits."""
    layers, hkv, idx, groups, new, ptok, hq, ballast = SHAPES[shape]
    s = Shared(pkv.layout(layers, hkv, 256, idx, fmt), groups, new, ptok, n_q_heads=hq, ballast=ballast)
    assert not decoded_alone(s, s.call())


@pytest.mark.parametrize("fmt", [BF, E4])
@pytest.mark.parametrize("ptok", [64, 128, 16])
@pytest.mark.parametrize("last", [False, True], ids=["before", "behind"])
def test_more_bases_than_a_call_has_maps(fmt, ptok, last):
    """Eighteen contiguous streams, each of a buffer of its own, before (behind) groups that share: the groups (the last streams) go key by key."""
    t, lay, hq, n = torch(), pkv.layout(1, 2, 256, 0, fmt), 8, 18
    a = Shared(lay, [([100 + 5 * i], 0) for i in range(n)], [1 + i % 3 for i in range(n)], ptok, n_q_heads=hq, seed=1)
    b = Shared(lay, [([33, 4, 150], 5), ([20, 21], 3)], 2, ptok, n_q_heads=hq, seed=2, ballast=24)
    buffers = [t.full((1, pkv.page_elems(lay, 192)), 0x7FC1, dtype=t.int16, device="cuda") for _ in range(n)]
    lone = []
    for i, x in enumerate(buffers):
        g, length = pkv.Pg(x.data_ptr(), None, x.shape[1], 192, 1, 1, 0), a.lens[i]
        pkv.store(lay, [pkv.seq(g, length, length)], 0, a.dev(a.k[i]), a.dev(a.v[i]))
        lone.append(pkv.seq(g, length, a.new[i]))
    order = (b, a) if last else (a, b)
    seqs = b.seqs + lone if last else lone + b.seqs
    groups = b.groups + a.groups if last else a.groups + b.groups
    q, st = t.cat([s.dq for s in order]), t.zeros(1, dtype=t.int32, device="cuda")
    ws = t.full((max(64, pkv.prefix_decode_ws_size(lay, seqs, groups, hq) // 4),), float("nan"), device="cuda")
    out = t.full((q.shape[0] + 1, hq, 256), 77, dtype=t.int16, device="cuda")
    pkv.prefix_decode(lay, seqs, groups, 0, hq, q, out, ws, status=st)
    assert int(st) == 0
    at = 0
    for s in order:
        s.check(t.cat([out[at:at + s.dq.shape[0]], out[-1:]]))
        at += s.dq.shape[0]


@pytest.mark.parametrize("fmt", [BF, E4])
def test_one_stream_left_stores_its_rows(fmt):
    """... beyond the windowed decode's workspace, with the new rows stored by the call: pages and bits as by a store before it."""
    t, lay = torch(), pkv.layout(1, 40, 256, 128, fmt)
    a, b = (Shared(lay, [([20, 9, 30], 11), ([30], 0)], [0, 2, 0, 1], 64, n_q_heads=40, fused=True) for _ in range(2))
    pkv.store(lay, b.seqs, 0, b.k_new, b.v_new, b.ik_new)
    b.fused = False
    one, two = a.call(), b.call()
    a.check(one)
    assert t.equal(a.mem, b.mem) and t.equal(one, two) and not decoded_alone(a, one)
