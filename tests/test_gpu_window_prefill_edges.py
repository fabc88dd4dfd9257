"""Windowed chunk attention at the edges of its inputs' range, against the
attention's definition in float64 (bound: gpu_setup.bound)."""
import numpy as np
import pytest

from paged_kv_cache_pg_gb300 import pkv

from gpu_setup import dev_u16, host_u16, torch, within_tol
from window_setup import Windowed, queries_of, streams_of

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    from paged_kv_cache_pg_gb300 import build
    build.build()
    pkv.load()


def run(w, hq, q_list, expect=0):
    t = torch()
    seqs = w.seqs()
    q = dev_u16(np.concatenate(q_list))
    out = t.zeros_like(q)
    status = t.zeros(1, dtype=t.int32, device="cuda")
    size = pkv.window_prefill_ws_size(w.lay, seqs, hq, w.window, w.sinks)
    ws = t.full((max(64, size // 4),), float("nan"), dtype=t.float32, device="cuda")
    pkv.window_prefill(w.lay, seqs, 0, hq, w.window, w.sinks, q, out, ws, status=status)
    assert int(status) == expect
    return host_u16(out)


def bf16_of(x):
    """bf16 bits of values that bf16 holds exactly."""
    f = np.asarray(x, np.float32)
    assert not (f.view(np.uint32) & 0xFFFF).any()
    return (f.view(np.uint32) >> 16).astype(np.uint16)


# (lens, n_new, window): one split; several
CALLS = [([300, 64], [70, 64], 100), ([2600], [20], 2400)]


@pytest.mark.parametrize("lens,n_new,window", CALLS)
@pytest.mark.parametrize("e", [0, 5, 8, 10, 12, 16, 24])
def test_large_scores(e, lens, n_new, window):
    # keys of -2 .. 2 and queries of -8 .. 8 times 2^e: every score is exact in
    # float32, up to 2^e x 27 after its scale, and ties are exact
    hq, hkv, sinks = 8, 2, 4
    lay = pkv.layout(1, hkv, 256, 0)
    rng = np.random.default_rng(e)
    ss = streams_of(lens, hkv, seed=3)
    for s in ss:
        s.k[0] = bf16_of(rng.integers(-2, 3, s.k[0].shape))
    q = [bf16_of(rng.integers(-8, 9, (n, hq, 256)) * 2.0 ** e) for n in n_new]
    w = Windowed(lay, ss, n_new, window, sinks, 16, seed=2)
    if e == 24:               # scores of some 10^8, which float32 cannot tell apart by one: reported
        run(w, hq, q, expect=pkv.DEV_RANGE)
        return
    ok, report = within_tol(run(w, hq, q), w.reference(0, q))
    assert ok, report


@pytest.mark.parametrize("lens,n_new,window", CALLS)
@pytest.mark.parametrize("shift", [-1.0, 1.0])
def test_scores_with_a_large_common_part(shift, lens, n_new, window):
    # keys that share a large component, which every query meets alike: scores
    # near +-250,000, 62,500 and a few after the scale
    hq, hkv, sinks = 4, 1, 4
    lay = pkv.layout(1, hkv, 256, 0)
    rng = np.random.default_rng(7)
    ss = streams_of(lens, hkv, seed=4)
    for s in ss:
        k = rng.integers(-2, 3, s.k[0].shape).astype(np.float32)
        k[..., 0] = 512.0 * shift
        s.k[0] = bf16_of(k)
    q = []
    for n in n_new:
        x = rng.integers(-2, 3, (n, hq, 256)).astype(np.float32)
        x[..., 0] = 496.0
        q.append(bf16_of(x))
    w = Windowed(lay, ss, n_new, window, sinks, 16, seed=2)
    ok, report = within_tol(run(w, hq, q), w.reference(0, q))
    assert ok, report
