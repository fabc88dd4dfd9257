"""Windowed chunk attention at the edges of its inputs' range, against the
attention's definition in float64 (bound: gpu_setup.bound)."""
import numpy as np
import pytest

from paged_kv_cache_pg_gb300 import pkv

from gpu_setup import dev_u16, host_u16, torch, within_tol
from window_setup import Windowed, attend, queries_of, streams_of, values

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


NAN, INF, NINF = 0x7FC1, 0x7F80, 0xFF80
# what KV head 0 of the first stream (or all queries of its heads) holds, as
# (tensor, position from the stream's end, dim, bits); every query reads it
BAD = [[("k", 50, 3, NAN)], [("v", 50, 3, NAN)], [("q", 0, 5, NAN)], [("k", 50, 3, INF)], [("q", 0, 5, INF)],
       [("v", 50, 3, INF), ("v", 40, 3, NINF)], [("k", p, 0, NAN) for p in range(1, 301)]]


@pytest.mark.parametrize("case", range(len(BAD)))
@pytest.mark.parametrize("lens,n_new,window", [([300, 64], [20, 64], 100), ([2600], [20], 2400)])
def test_what_is_not_finite_where_it_is_read_is_not_finite_in_the_output(lens, n_new, window, case):
    hq, hkv, sinks = 8, 2, 4
    grp = hq // hkv
    lay = pkv.layout(1, hkv, 256, 0)
    ss = streams_of(lens, hkv, seed=61)
    q = queries_of(n_new, hq, seed=62)
    clean = Windowed(lay, ss, n_new, window, sinks, 16, seed=5).reference(0, q)
    for what, back, dim, bits in BAD[case]:
        if what == "q":
            q[0][:, :grp, dim] = bits
        else:
            getattr(ss[0], what)[0][lens[0] - back, 0, dim] = bits
    got = run(Windowed(lay, ss, n_new, window, sinks, 16, seed=5), hq, q, expect=pkv.DEV_RANGE)
    with np.errstate(all="ignore"):
        want = attend(values(ss[0].k[0], 0), values(ss[0].v[0], 0), q[0], lens[0], window, sinks)
    n = n_new[0]
    odd = (got[:n, :grp] & 0x7F80) == 0x7F80
    assert np.array_equal(odd, ~np.isfinite(want[:, :grp])) and odd.any()
    rest = np.concatenate([got[:n, grp:].ravel(), got[n:].ravel()])
    ok, report = within_tol(rest, np.concatenate([clean[:n, grp:].ravel(), clean[n:].ravel()]))
    assert ok, report
