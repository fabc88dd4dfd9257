"""Windowed decode at the edges of its plan and of its inputs' range, against the
attention's definition in float64 (bound: gpu_setup.bound)."""
import numpy as np
import pytest

from paged_kv_cache_pg_gb300 import pkv, synth

from gpu_setup import dev_u16, host_u16, torch, within_tol
from window_setup import Windowed, queries_of, streams_of

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
