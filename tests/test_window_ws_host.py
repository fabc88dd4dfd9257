"""The windowed decode's workspace near the window lengths where a split is
added: the size for the longest length and the most new tokens covers every
shorter one, and no call needs more than it says.  No GPU needed."""
import numpy as np
import pytest

from paged_kv_cache_pg_gb300 import build, pkv


@pytest.fixture(scope="module", autouse=True)
def lib():
    build.build()
    return pkv.load()


CAP = 21000


def _size(lay, lens, new, hq, window, sinks):
    page = pkv.pg(1 << 20, None, pkv.page_elems(lay, CAP), CAP)
    return pkv.window_decode_ws_size(lay, [pkv.seq(page, int(n), int(m)) for n, m in zip(lens, new)], hq, window, sinks)


FMT = [pkv.KV_BF16, pkv.KV_E4M3]


@pytest.mark.parametrize("fmt", FMT)
@pytest.mark.parametrize("sinks", [0, 4, 17, 64])
@pytest.mark.parametrize("border", [5120, 10240, 15360])
def test_one_stream_at_every_length_of_two_tiles(border, sinks, fmt):
    lay = pkv.layout(1, 2, 256, 0, fmt)
    for window in range(border - sinks - 80, border - sinks + 24):
        for top in (20000, 20011, 19990):
            most = _size(lay, [top], [2], 16, window, sinks)
            sizes = [_size(lay, [n], [m], 16, window, sinks) for m in (1, 2)
                     for n in [*range(top - 40, top + 1, 3), window - 1, window + sinks, window + sinks + 15, window + sinks + 31]]
            assert max(sizes) <= most, (window, top)


@pytest.mark.parametrize("fmt", FMT)
def test_sizes_grow_with_the_length_and_the_new_tokens(fmt):
    lay = pkv.layout(1, 1, 256, 0, fmt)
    for window, sinks in ((5100, 4), (5090, 9), (10236, 4), (2560, 2550), (60, 5050)):
        last = 0
        for n in [*range(1, 200, 7), *range(2400, 2800, 5), *range(5000, 5400, 3), *range(10100, 10500, 5), 20000]:
            sizes = [_size(lay, [n], [min(n, m)], 8, window, sinks) for m in (0, 1, 2, 4)]
            assert sizes == sorted(sizes) and sizes[-1] >= last, (window, sinks, n)
            last = sizes[-1]


@pytest.mark.parametrize("fmt", FMT)
@pytest.mark.parametrize("streams,hq,window", [(24, 16, 5106), (64, 16, 5090), (9, 32, 10230), (40, 8, 5060)])
def test_batches_near_a_border(fmt, streams, hq, window):
    rng = np.random.default_rng(streams)
    lay = pkv.layout(1, 2, 256, 0, fmt)
    top_new = max(1, 32 // (hq // 2))
    most = _size(lay, [20000] * streams, [top_new] * streams, hq, window, 4)
    for _ in range(100):
        lens = rng.integers(window - 40, 20001, streams)
        assert _size(lay, lens, rng.integers(0, top_new + 1, streams), hq, window, 4) <= most
