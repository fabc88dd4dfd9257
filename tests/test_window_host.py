"""Windowed attention: its refusals, workspace sizes and dead pages, without a GPU."""
import ctypes

import numpy as np
import pytest

from paged_kv_cache_pg_gb300 import build, pkv


@pytest.fixture(scope="module", autouse=True)
def lib():
    build.build()
    return pkv.load()


def _seq(lay, length=600, n_new=1, ptok=16, n_table=50, n_pages=64, base=0x10000):
    return pkv.seq(pkv.Pg(base, 0x20000, pkv.page_elems(lay, ptok), ptok, n_pages, n_table, 0), length, n_new)


def _call(lay, seqs, window=100, n_sink=4, hq=4, layer=0, q=0x1000, out=0x1000, k=None, v=None, ik=None, ws=None,
          ws_bytes=0):
    arr, n = pkv._seqs(seqs)
    return pkv.load().pkv_window_decode(ctypes.byref(lay), arr, n, layer, hq, window, n_sink, q, k, v, ik, out, ws,
                                        ws_bytes, None, None)


def _ws(lay, seqs, window, n_sink, hq=4):
    return pkv.window_decode_ws_size(lay, seqs, hq, window, n_sink)


@pytest.mark.parametrize("fmt", [pkv.KV_BF16, pkv.KV_E4M3])
def test_refusals_before_launch(fmt):
    lay = pkv.layout(2, 2, 256, 128, fmt)
    s = _seq(lay)
    for kw in (dict(window=0), dict(window=-5), dict(n_sink=-1), dict(hq=3), dict(layer=2), dict(q=None), dict(out=None),
               dict(q=0x1008), dict(out=0x1008), dict(k=0x1000), dict(v=0x1000), dict(k=0x1000, v=0x1000),
               dict(k=0x1000, v=0x1000, ik=0x1008), dict(k=0x1008, v=0x1000, ik=0x1000), dict(hq=66)):
        assert _call(lay, [s], **kw) == pkv.EINVAL, kw
    assert _call(lay, [_seq(lay, n_new=17)]) == pkv.EINVAL            # 34 query columns
    assert _call(lay, [_seq(lay, length=801)]) == pkv.EINVAL          # past the table
    assert _call(lay, [_seq(lay, n_new=601)]) == pkv.EINVAL
    assert _call(lay, [s] * 65) == pkv.EINVAL
    assert _call(lay, []) == pkv.OK                                    # nothing launched
    assert _call(lay, [_seq(lay, n_new=0), _seq(lay, length=0, n_new=0)]) == pkv.OK
    out = ctypes.c_size_t()
    arr, n = pkv._seqs([s])
    assert pkv.load().pkv_window_decode_ws_size(ctypes.byref(lay), arr, n, 4, 0, 0, ctypes.byref(out)) == pkv.EINVAL
    assert pkv.load().pkv_window_decode_ws_size(ctypes.byref(lay), arr, n, 4, 1, 0, None) == pkv.EINVAL


def test_short_windows_need_no_workspace_and_long_ones_are_checked():
    lay = pkv.layout(1, 2)
    s = _seq(lay, length=40000, ptok=256, n_table=200, n_pages=200)
    assert _ws(lay, [s], 4096, 64) == 0
    need = _ws(lay, [s], 20000, 4)
    assert need > 0
    assert _ws(lay, [s, s], 20000, 4) == 2 * need
    assert _call(lay, [s], 20000) == pkv.EINVAL
    assert _call(lay, [s], 20000, ws=0x1000, ws_bytes=need - 4) == pkv.EINVAL
    assert _call(lay, [s], 20000, ws=0x1080, ws_bytes=need) == pkv.EINVAL
    # the largest window and sink counts do not overflow
    assert _ws(lay, [s], 2**31 - 1, 2**31 - 1) == _ws(lay, [s], 40000, 0)


def test_dead_pages_are_exactly_those_no_later_query_reads():
    rng = np.random.default_rng(2)
    for _ in range(400):
        ptok = int(rng.choice([4, 16, 20, 48]))
        length, window, sinks = (int(rng.integers(0, 300)), int(rng.integers(1, 120)), int(rng.integers(0, 70)))
        first, end = pkv.window_dead_pages(ptok, length, window, sinks)
        j = np.arange(0, length + ptok)
        read = (j < sinks) | (j > length - window)
        dead = [p for p in range(length // ptok + 1) if not read[p * ptok:(p + 1) * ptok].any()]
        assert list(range(first, end)) == dead, (ptok, length, window, sinks)
    assert pkv.window_dead_pages(16, 1000, 2**31 - 1, 0) == (0, 0)
    a, b = pkv.window_dead_pages(16, 1000, 1, 2**31 - 1)
    assert a == b
    for bad in ((18, 1, 1, 0), (0, 1, 1, 0), (16, -1, 1, 0), (16, 1, 0, 0), (16, 1, 1, -1)):
        with pytest.raises(pkv.PkvError) as e:
            pkv.window_dead_pages(*bad)
        assert e.value.code == pkv.EINVAL


def test_calls_take_only_contiguous_tensors_of_the_device():
    import torch
    lay = pkv.layout(1, 1, 256, 0)
    with pytest.raises(pkv.PkvError) as e:
        pkv.window_decode(lay, [_seq(lay)], 0, 4, 100, 4, torch.zeros(4, 256, dtype=torch.bfloat16), 0x1000, stream=0)
    assert e.value.code == pkv.EINVAL


# ---- the chunk form ------------------------------------------------------------

def _chunk(lay, seqs, window=100, n_sink=4, hq=4, layer=0, q=0x1000, out=0x1000, ws=0x1000, ws_bytes=1 << 40):
    arr, n = pkv._seqs(seqs)
    return pkv.load().pkv_window_prefill(ctypes.byref(lay), arr, n, layer, hq, window, n_sink, q, out, ws, ws_bytes,
                                         None, None)


def test_chunk_refusals_before_launch():
    # with a stream that has queries the call asks for the SM count before it
    # checks its pointers: every answer here is a refusal either way
    lay = pkv.layout(2, 2, 256, 128)
    s = _seq(lay, n_new=30)
    for kw in (dict(window=0), dict(window=-1), dict(n_sink=-1), dict(hq=3), dict(layer=2)):
        assert _chunk(lay, [s], **kw) == pkv.EINVAL, kw
    assert _chunk(pkv.layout(2, 2, 256, 128, pkv.KV_E4M3), [_seq(pkv.layout(2, 2, 256, 128, pkv.KV_E4M3))]) == pkv.EINVAL
    for kw in (dict(q=None), dict(out=None), dict(q=0x1008), dict(out=0x1008), dict(ws=None), dict(ws=0x1080), dict(ws_bytes=64)):
        assert _chunk(lay, [s], **kw) != pkv.OK, kw
    assert _chunk(lay, [_seq(lay, n_new=601)]) == pkv.EINVAL
    assert _chunk(lay, [_seq(lay, length=801, n_new=30)]) == pkv.EINVAL
    assert pkv.load().pkv_window_prefill_ws_size(ctypes.byref(lay), pkv._seqs([s])[0], 1, 4, 100, 4, None) == pkv.EINVAL


@pytest.mark.parametrize("fmt", [pkv.KV_BF16, pkv.KV_E4M3])
@pytest.mark.parametrize("streams,hq,window", [(24, 16, 4096), (64, 16, 512), (7, 8, 9000), (64, 64, 60), (40, 16, 2047)])
def test_the_workspace_of_the_longest_lengths_covers_shorter_ones(fmt, streams, hq, window):
    rng = np.random.default_rng(streams + hq)
    lay = pkv.layout(1, 2 if hq < 64 else 4, 256, 0, fmt)
    group = hq // lay.n_kv_heads

    def size(lens, new):
        page = pkv.pg(1 << 20, None, pkv.page_elems(lay, 20000), 20000)
        return pkv.window_decode_ws_size(lay, [pkv.seq(page, int(n), int(m)) for n, m in zip(lens, new)], hq, window, 4)

    top_new = max(1, 32 // group)
    most = size([20000] * streams, [top_new] * streams)
    for _ in range(200):
        lens = np.exp(rng.uniform(np.log(top_new), np.log(20000), streams)).astype(int).clip(top_new)
        assert size(lens, rng.integers(0, top_new + 1, streams)) <= most


def test_more_queries_or_positions_than_32_bits_count_are_refused():
    # 2^28 new tokens of 16 heads a KV head: 2^32 query columns; a stream of 2^29 + 4 positions
    lay = pkv.layout(1, 1, 256, 0)
    for length, n_new in ((1 << 28, 1 << 28), ((1 << 29) + 4, 1)):
        seqs = [pkv.seq(pkv.Pg(0x10000, 0, pkv.page_elems(lay, length), length, 1, 0, 0), length, n_new)]
        for size in (pkv.window_decode_ws_size, pkv.window_prefill_ws_size):
            with pytest.raises(pkv.PkvError) as e:
                size(lay, seqs, 16, 100, 0)
            assert e.value.code == pkv.EINVAL
