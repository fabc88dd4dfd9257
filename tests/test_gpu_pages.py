"""Page copies and table rewrites on the GPU, byte for byte, and a run of
them as a server would use them: fork, decode both, compact, decode again."""
import numpy as np
import pytest

from paged_kv_cache_pg_gb300 import pkv, synth

from gpu_setup import GUARD, dev_u16, host_u16, place, torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    from paged_kv_cache_pg_gb300 import build
    build.build()
    pkv.load()


def _random_arena(lay, ptok, n_pages, seed):
    t = torch()
    ps = pkv.page_elems(lay, ptok)
    host = np.random.default_rng(seed).integers(0, 1 << 16, n_pages * ps + 2 * GUARD, dtype=np.uint16)
    buf = dev_u16(host)
    return ps, host[GUARD:GUARD + n_pages * ps].reshape(n_pages, ps).copy(), buf, buf[GUARD:GUARD + n_pages * ps]


def _bytes_of(lay, ptok, n_pos):
    """Mask of a page's bytes that belong to its first n_pos positions, from
    the host's row addresses."""
    ps = pkv.page_elems(lay, ptok)
    mask = np.zeros(2 * ps, bool)
    g = pkv.pg(0x10000, None, ps, ptok)
    fp8 = lay.kv_format == pkv.KV_E4M3
    unit = 1 if fp8 else 2                     # pg_row counts bytes for e4m3, elements else
    kinds = [(pkv.K, 256 * unit), (pkv.V, 256 * unit)]
    if fp8:
        kinds += [(pkv.KS, 4), (pkv.VS, 4)]
    for layer in range(lay.n_layers):
        for kind, size in kinds:
            for head in range(lay.n_kv_heads):
                for pos in range(n_pos):
                    at = unit * pkv.pg_row(lay, g, None, layer, kind, head, pos)
                    mask[at:at + size] = True
        if lay.idx_dim:
            for kind, rows in ((pkv.IK, n_pos), (pkv.P, n_pos // 4)):
                for pos in range(rows):
                    at = unit * pkv.pg_row(lay, g, None, layer, kind, 0, pos)
                    mask[at:at + 2 * lay.idx_dim] = True
    return mask


LAYOUTS = [(1, 1, 0, pkv.KV_BF16), (3, 2, 128, pkv.KV_BF16), (1, 1, 0, pkv.KV_E4M3), (2, 3, 128, pkv.KV_E4M3)]


@pytest.mark.parametrize("layers,hkv,idx,fmt", LAYOUTS)
@pytest.mark.parametrize("ptok", [4, 20, 64])
def test_copies_move_exactly_the_positions_asked_for(layers, hkv, idx, fmt, ptok):
    lay = pkv.layout(layers, hkv, 256, idx, fmt)
    n_pages = 14
    ps, want, buf, body = _random_arena(lay, ptok, n_pages, ptok + layers)
    before = host_u16(buf).copy()
    src, dst = [9, 3, 3, 0, 13, 9, 1], [2, 4, 5, 6, 7, 8, 10]
    n_pos = [ptok, 1, ptok - 1, 0, 3, min(ptok, 4), ptok // 2 + 1]
    pkv.pages_copy(lay, ptok, body, n_pages, src, dst, n_pos=n_pos)
    w = want.view(np.uint8).reshape(n_pages, -1)
    for s, d, n in zip(src, dst, n_pos):
        m = _bytes_of(lay, ptok, n)
        w[d][m] = w[s][m]
    got = host_u16(buf)
    assert np.array_equal(got[GUARD:-GUARD].reshape(n_pages, ps), want)
    assert np.array_equal(got[:GUARD], before[:GUARD]) and np.array_equal(got[-GUARD:], before[-GUARD:])


@pytest.mark.parametrize("fmt", [pkv.KV_BF16, pkv.KV_E4M3])
def test_more_copies_than_one_launch_takes(fmt):
    lay = pkv.layout(1, 1, 256, 128, fmt)
    n_pages = 2500
    ps, want, buf, body = _random_arena(lay, 4, n_pages, 5)
    perm = np.random.default_rng(1).permutation(n_pages).astype(np.int32)
    src, dst = perm[:1200], perm[1200:2400]
    pkv.pages_copy(lay, 4, body, n_pages, src, dst)
    want[dst] = want[src]
    assert np.array_equal(host_u16(body).reshape(n_pages, ps), want)


def test_copy_beyond_four_gigabytes():
    t = torch()
    lay = pkv.layout(13, 2, 256, 128)
    ps = pkv.page_elems(lay, 256)
    n_pages = 600                                        # 4.7 GB: byte offsets pass 32 bits
    mem = t.zeros(n_pages * ps, dtype=t.int16, device="cuda").view(n_pages, ps)
    mem[0].random_(-30000, 30000)
    mem[598].random_(-30000, 30000)
    pkv.pages_copy(lay, 256, mem, n_pages, [0, 598], [599, 1], n_pos=[256, 100])
    assert t.equal(mem[599], mem[0])
    m = t.from_numpy(_bytes_of(lay, 256, 100)[::2].copy()).cuda()
    assert t.equal(mem[1][m], mem[598][m]) and not mem[1][~m].any() and not mem[2:598].any()


@pytest.mark.parametrize("n_tables,size,n_moves", [(1, 1, 1), (3, 257, 40), (70, 33, 1300)])
def test_tables_are_rewritten_and_other_entries_stay(n_tables, size, n_moves):
    t = torch()
    rng = np.random.default_rng(n_moves)
    perm = rng.permutation(2 * n_moves + 50).astype(np.int32)
    src, dst = perm[:n_moves], perm[n_moves:2 * n_moves]
    host = rng.integers(-3, perm.size, (n_tables, size + 2)).astype(np.int32)
    dev = t.from_numpy(host).cuda()
    pkv.tables_remap([d[1:-1] for d in dev] + [dev[0][1:-1], dev[0][:0]], src, dst)
    to = np.arange(-3, perm.size, dtype=np.int32)
    to[src + 3] = dst
    want = host.copy()
    want[:, 1:-1] = to[host[:, 1:-1] + 3]
    assert np.array_equal(dev.cpu().numpy(), want)


def test_copy_and_remap_are_captured_and_replayed():
    t = torch()
    lay = pkv.layout(1, 1, 256, 0)
    ps = pkv.page_elems(lay, 16)
    mem = t.zeros(6, ps, dtype=t.int16, device="cuda")
    table = t.tensor([4, 5, 1], dtype=t.int32, device="cuda")
    g = t.cuda.CUDAGraph()
    with t.cuda.graph(g):
        pkv.pages_copy(lay, 16, mem, 6, [4, 5], [0, 2])
        pkv.tables_remap([table], [4, 5], [0, 2])
    for k in range(2):
        mem[4], mem[5] = 7 + k, 9 + k
        table.copy_(t.tensor([4, 5, 1], dtype=t.int32))
        g.replay()
        assert (mem[0] == 7 + k).all() and (mem[2] == 9 + k).all()
        assert table.tolist() == [0, 2, 1]


def _decode(lay, g, length, hq, q, status):
    t = torch()
    seqs = [pkv.seq(g, length, 1)]
    out = t.zeros_like(q)
    ws = t.zeros(max(64, pkv.decode_ws_size(lay, seqs, hq) // 4 + 64), dtype=t.float32, device="cuda")
    pkv.decode(lay, seqs, 0, hq, q, out, ws, status=status)
    return out


def test_fork_then_compact_keeps_every_stream_s_output():
    t = torch()
    lay = pkv.layout(2, 2, 256, 128)
    ptok, T, hq = 16, 150, 4
    n_pages = 30
    ps = pkv.page_elems(lay, ptok)
    mem = t.full((n_pages * ps,), 0x7FC1, dtype=t.int16, device="cuda")
    a = pkv.Arena(lay, ptok, mem)
    hole = a.take(7)
    ids = a.take(-(-T // ptok))
    a.give(hole, defer=False)
    s = synth.make_stream(1, 2, T + 8, 2, 256, 128)
    table = t.from_numpy(ids.copy()).cuda()
    g = a.pg(table)
    for layer in range(2):
        pkv.store(lay, [pkv.seq(g, T, T)], layer, dev_u16(s.k[layer][:T]), dev_u16(s.v[layer][:T]), dev_u16(s.ik[layer][:T]))
    # the fork: shared whole pages, its own copy of the last one
    fids, copy = a.fork(ids, T)
    ftable = t.from_numpy(fids.copy()).cuda()
    fg = a.pg(ftable)
    pkv.pages_copy(lay, ptok, mem, n_pages, [copy[0]], [copy[1]], n_pos=[copy[2]])
    status = t.zeros(1, dtype=t.int32, device="cuda")
    q = dev_u16(synth.queries(2, 1, hq, 256))
    base = _decode(lay, g, T, hq, q, status)
    assert t.equal(base, _decode(lay, fg, T, hq, q, status))
    # both go on with other tokens: neither sees the other's
    for stream, at in ((g, 0), (fg, 4)):
        pkv.store(lay, [pkv.seq(stream, T + 4, 4)], 0, *(dev_u16(x[0][T + at:T + at + 4]) for x in (s.k, s.v, s.ik)))
    one, two = _decode(lay, g, T + 4, hq, q, status), _decode(lay, fg, T + 4, hq, q, status)
    alone = pkv.page_elems(lay, 160)
    for at, got in ((0, one), (4, two)):
        buf = t.zeros(alone, dtype=t.int16, device="cuda")
        cg = pkv.pg(buf, None, alone, 160)
        rows = [np.concatenate([x[0][:T], x[0][T + at:T + at + 4]]) for x in (s.k, s.v, s.ik)]
        pkv.store(lay, [pkv.seq(cg, T + 4, T + 4)], 0, *(dev_u16(r) for r in rows))
        assert t.equal(got, _decode(lay, cg, T + 4, hq, q, status))
    # compaction: the copies, the tables, and a decode right behind them
    src, dst = a.compact(100)
    assert src.size == 6                                 # ids 1 .. 6 are free, the fork has 0
    pkv.pages_copy(lay, ptok, mem, n_pages, src, dst)
    pkv.tables_remap([table, ftable], src, dst)
    again = [_decode(lay, x, T + 4, hq, q, status) for x in (g, fg)]
    a.give(src)
    t.cuda.synchronize()
    assert t.equal(again[0], one) and t.equal(again[1], two) and int(status) == 0
    to = np.arange(n_pages)
    to[src] = dst
    assert table.tolist() == to[ids].tolist() and ftable.tolist() == to[fids].tolist()
    assert max(table.tolist() + ftable.tolist()) < 11 and a.info()[1] == n_pages - 11
    a.give(to[ids], defer=False)
    a.give(to[fids], defer=False)
    assert a.info()[1] == n_pages
