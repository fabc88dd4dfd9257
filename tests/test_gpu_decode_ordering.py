"""Decode calls that store their new rows, one directly behind the other on one
stream and layer: each reads cached rows more than 32 below its new tokens before
the calls in front of it have finished, up to 32 rows a call back.  Captured and
replayed without a wait, against the same calls with a wait after each."""
import pytest

from paged_kv_cache_pg_gb300 import pkv

from gpu_setup import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    from paged_kv_cache_pg_gb300 import build
    build.build()
    pkv.load()


# new tokens of the calls in turn, of one query head a KV head: bf16 calls of more
# than 16 take the tensor-core route
STEPS = [[32], [16], [1], [20, 1, 1, 13], [32, 1], [17, 16, 3]]


@pytest.mark.parametrize("fmt", [pkv.KV_BF16, pkv.KV_E4M3])
@pytest.mark.parametrize("kind", ["decode", "mixed"])
@pytest.mark.parametrize("steps", STEPS, ids=str)
@pytest.mark.parametrize("streams", [1, 3])
def test_storing_calls_follow_each_other_directly(steps, streams, kind, fmt):
    t = torch()
    T, hkv, ptok = 640, 2, 16
    lay = pkv.layout(1, hkv, 256, 0, fmt)
    ps, per = pkv.page_elems(lay, ptok), T // ptok
    g = t.Generator(device="cuda").manual_seed(5)
    tables = t.randperm(per * streams, device="cuda", generator=g).to(t.int32).view(streams, per)
    calls, at = [], 0
    while at + max(steps) <= T and len(calls) < 120:
        n = steps[len(calls) % len(steps)]
        rows = [t.randn(streams * n, hkv, 256, device="cuda", generator=g).to(t.bfloat16) for _ in range(3)]
        calls.append((at, n, rows))
        at += n
    mem = t.full((per * streams, ps), 0x7FC1, dtype=t.int16, device="cuda")
    status = t.zeros(1, dtype=t.int32, device="cuda")
    work = []
    for i, (at, n, (k, v, q)) in enumerate(calls):
        seqs = pkv.batch([pkv.seq(pkv.pg(mem, x, ps, ptok, per * streams), at + n, n) for x in tables])
        size = pkv.decode_ws_size(lay, seqs, hkv)
        ws = t.zeros(max(64, size // 4 + 64), dtype=t.float32, device="cuda")
        work.append((seqs, k, v, q, t.zeros_like(q), ws))

    def run(wait):
        for i, (seqs, k, v, q, out, ws) in enumerate(work):
            if kind == "mixed" and i % 3 == 2:
                pkv.window_decode(lay, seqs, 0, hkv, 10 ** 6, 0, q, out, None, status=status, k_new=k, v_new=v)
            else:
                pkv.decode(lay, seqs, 0, hkv, q, out, ws, status=status, k_new=k, v_new=v)
            if wait:
                t.cuda.synchronize()

    run(True)
    t.cuda.synchronize()
    want = [w[4].clone() for w in work], mem.clone()
    assert all(x.isfinite().all() for x in want[0])
    graph = t.cuda.CUDAGraph()
    with t.cuda.graph(graph):
        run(False)
    for _ in range(8):
        mem.fill_(0x7FC1)
        for w in work:
            w[4].zero_()
        graph.replay()
        t.cuda.synchronize()
        assert all(t.equal(w[4], x) for w, x in zip(work, want[0])) and t.equal(mem, want[1])
    assert int(status) == 0
