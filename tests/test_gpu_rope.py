"""Rotary positions on the GPU against their definition in float64, alone and on the way into the pages."""
import numpy as np
import pytest

import oracle as orc
from paged_kv_cache_pg_gb300 import pkv

import rope_setup as rs
from gpu_setup import torch

pytestmark = pytest.mark.gpu

HALF, INTER = pkv.ROPE_HALF, pkv.ROPE_INTERLEAVED
BF16_STEP = 2.0 ** -8    # a rounding to bf16, relative to the value


@pytest.fixture(scope="module", autouse=True)
def built():
    from paged_kv_cache_pg_gb300 import build
    build.build()
    pkv.load()


def dev(bits):
    return torch().from_numpy(np.ascontiguousarray(bits).view(np.int16)).cuda()


def host(t):
    return t.cpu().numpy().view(np.uint16)


def seqs_of(lens):
    return [pkv.seq(pkv.Pg(), n, m) for n, m in lens]


def places(lens):
    return np.concatenate([np.arange(n - m, n) for n, m in lens] or [np.zeros(0, int)])


def close(got_bits, want, size):
    got = rs.bf16_values(got_bits)
    assert (np.abs(got - want) <= BF16_STEP * np.abs(want) + rs.slack(size)).all(), np.abs(got - want).max()


@pytest.mark.parametrize("pairs", [HALF, INTER])
@pytest.mark.parametrize("dim,rot", [(256, 256), (256, 64), (256, 2), (256, 6), (256, 20), (256, 250), (128, 128), (128, 32), (128, 14)])
@pytest.mark.parametrize("heads,lens", [(1, [(1, 1)]), (16, [(9001, 1), (7, 7), (500, 0), (40956, 3)]), (5, [(700, 1)])])
def test_rows(pairs, dim, rot, heads, lens):
    rng = np.random.default_rng(rot + heads)
    pos = places(lens)
    x = rs.random_rows(rng, len(pos), heads, dim)
    r = pkv.rope(rot, 1e4, pairs)
    f, scale = rs.freqs(rot, 1e4)
    out = torch().full((len(pos) + 1, heads, dim), 77, dtype=torch().int16, device="cuda")
    pkv.rope_rows(r, seqs_of(lens), heads, dev(x), out)
    want, size = rs.turn(rs.bf16_values(x), pos, rot, pairs, f, scale)
    got = host(out)
    close(got[:-1], want, size)
    assert np.array_equal(got[:-1][..., rot:], x[..., rot:]) and (got[-1] == 77).all()


def test_many_tokens_take_four_a_block():
    rng = np.random.default_rng(1)
    lens = [(3001, 2999), (17, 1)]
    pos = places(lens)
    x = rs.random_rows(rng, len(pos), 3, 256)
    out = torch().empty((len(pos), 3, 256), dtype=torch().int16, device="cuda")
    pkv.rope_rows(pkv.rope(128, 5e5, INTER, pkv.ROPE_BANDS, factor=8.0, original=8192), seqs_of(lens), 3, dev(x), out)
    f, scale = rs.freqs(128, 5e5, "bands", 8.0, 8192)
    close(host(out), *rs.turn(rs.bf16_values(x), pos, 128, INTER, f, scale))


def test_far_and_negative_positions_given():
    """Positions of the program's own: to the ends of int32 (whole turns go away exactly), and back again."""
    rng = np.random.default_rng(2)
    pos = np.array([2 ** 31 - 1, -2 ** 31, 10 ** 9 + 7, 0, -1, 123456789], np.int32)
    x = rs.random_rows(rng, len(pos), 2, 128)
    r = pkv.rope(128, 1e4, HALF, pkv.ROPE_YARN, factor=4.0, original=4096, scale=1.0)
    # the turns as the rope holds them, in whole numbers: an angle in float64 has lost 2^-22 of a radian at these positions
    turns = [[(int(t) * int(p)) % 2 ** 64 / 2.0 ** 64 for t in r.turns[:64]] for p in pos]
    out = torch().empty((len(pos), 2, 128), dtype=torch().int16, device="cuda")
    place = torch().from_numpy(pos).cuda()
    pkv.rope_rows(r, seqs_of([(6, 6)]), 2, dev(x), out, pos=place)
    v = rs.bf16_values(x)
    c, s = (fn(2 * np.pi * np.array(turns))[:, None] for fn in (np.cos, np.sin))
    want = np.concatenate([v[..., :64] * c - v[..., 64:] * s, v[..., 64:] * c + v[..., :64] * s], -1)
    size = np.tile(np.abs(v[..., :64]) + np.abs(v[..., 64:]), 2)
    close(host(out), want, size)
    # by the opposite positions the rows come back, two roundings off
    back = torch().empty_like(out)
    pkv.rope_rows(r, seqs_of([(6, 6)]), 2, out, back, pos=-place.clamp(min=-2 ** 31 + 1))
    got, keep = rs.bf16_values(host(back)), pos != -2 ** 31
    assert (np.abs(got - v)[keep] <= (BF16_STEP * (np.abs(v) + 2 * size) + 2 * rs.slack(size))[keep]).all()


def test_the_gradient_is_the_rotation_back():
    """<g, R x> = <R^T g, x> with R^T the rotation by -p: against differences of the forward pass in float64."""
    rng = np.random.default_rng(3)
    pos = np.array([5, 70, 3000], np.int32)
    f, scale = rs.freqs(64, 1e4)
    x, g = (rs.bf16_values(rs.random_rows(rng, 3, 1, 128)) for _ in range(2))
    loss = lambda y: (rs.turn(y, pos, 64, HALF, f, scale)[0] * g).sum()  # noqa: E731
    want = np.zeros_like(x)
    for i in np.ndindex(*x.shape):
        step = np.zeros_like(x)
        step[i] = 0.5
        want[i] = loss(x + step) - loss(x - step)      # linear: exact up to float64
    out = torch().empty((3, 1, 128), dtype=torch().int16, device="cuda")
    pkv.rope_rows(pkv.rope(64, 1e4), seqs_of([(3, 3)]), 1, dev(rs.bf16_bits(g)), out, pos=torch().from_numpy(-pos).cuda())
    close(host(out), want, rs.turn(g, -pos, 64, HALF, f, scale)[1])


@pytest.mark.parametrize("heads,dim,tokens", [(64, 256, 3), (65, 256, 2), (130, 128, 2), (200, 256, 1), (24, 256, 2100), (40, 128, 2053)])
def test_many_heads(heads, dim, tokens):
    """More heads than a CTA takes, and blocks of two and four tokens."""
    rng = np.random.default_rng(heads)
    lens = [(tokens + 70, tokens)]
    x = rs.random_rows(rng, tokens, heads, dim)
    out = torch().empty((tokens, heads, dim), dtype=torch().int16, device="cuda")
    pkv.rope_rows(pkv.rope(64, 1e4), seqs_of(lens), heads, dev(x), out)
    f, scale = rs.freqs(64, 1e4)
    close(host(out), *rs.turn(rs.bf16_values(x), places(lens), 64, HALF, f, scale))


@pytest.mark.parametrize("hkv,hq,tokens", [(64, 64, 5), (2, 130, 2), (33, 66, 3), (2, 16, 2200), (4, 16, 2050)])
def test_store_with_many_heads(hkv, hq, tokens):
    rng = np.random.default_rng(hkv)
    lay, lens = pkv.layout(1, hkv, 256, 128), [(tokens + 9, tokens)]
    a, b = Pages(lay, lens, 16, 1), Pages(lay, lens, 16, 1)
    q, k, v = (dev(rs.random_rows(rng, tokens, h, 256)) for h in (hq, hkv, hkv))
    ik, r = dev(rs.random_rows(rng, tokens, 128)), pkv.rope(64, 1e4, INTER)
    k2, q2 = torch().empty_like(k), torch().empty_like(q)
    pkv.rope_rows(r, b.seqs, hkv, k, k2)
    pkv.rope_rows(r, b.seqs, hq, q, q2)
    pkv.store(lay, b.seqs, 0, k2, v, ik)
    pkv.rope_store(lay, a.seqs, 0, r, k, v, ik, n_q_heads=hq, q=q, q_out=q)      # in place
    assert torch().equal(a.mem, b.mem) and torch().equal(q, q2)


@pytest.mark.parametrize("fmt", [pkv.KV_BF16, pkv.KV_E4M3])
@pytest.mark.parametrize("given", [False, True])
def test_a_large_call_is_its_small_ones(fmt, given):
    """Units one after another in a CTA: the bits of calls of a CTA a token, positions of the cache's or given."""
    rng, t = np.random.default_rng(21), torch()
    lay, lens = pkv.layout(1, 2, 256, 128, fmt), [(6100, 6003), (3000, 2998), (40, 2)]
    a, b = Pages(lay, lens, 48, 1), Pages(lay, lens, 48, 1)
    tokens = sum(m for _, m in lens)
    q, k, v = (dev(rs.random_rows(rng, tokens, h, 256)) for h in (6, 2, 2))
    ik, r = dev(rs.random_rows(rng, tokens, 128)), pkv.rope(64, 1e4)
    pos = t.randint(-50000, 50000, (tokens,), dtype=t.int32, device="cuda") if given else None
    out, rows, small = t.empty_like(q), t.empty_like(q), t.empty_like(q)
    pkv.rope_store(lay, a.seqs, 0, r, k, v, ik, n_q_heads=6, q=q, q_out=out, pos=pos)
    pkv.rope_rows(r, a.seqs, 6, q, rows, pos=pos)
    at = 0
    for g, (n, m) in zip([x.pg for x in b.seqs], lens):
        for first in range(0, m, 1000):
            step = min(1000, m - first)
            s = slice(at + first, at + first + step)
            pkv.rope_store(lay, [pkv.seq(g, n - m + first + step, step)], 0, r, k[s], v[s], ik[s], n_q_heads=6, q=q[s], q_out=small[s],
                           pos=pos[s] if given else None)
        at += m
    assert t.equal(a.mem, b.mem) and t.equal(out, small) and t.equal(rows, small)


@pytest.mark.parametrize("pairs,rot", [(HALF, 256), (HALF, 20), (INTER, 64)])
def test_in_place_and_strided_rows(pairs, rot):
    rng = np.random.default_rng(4)
    n, heads, wide = 9, 6, 6 * 256 + 512 + 8
    flat = rs.random_rows(rng, n, wide)
    r, s = pkv.rope(rot, 1e4, pairs), seqs_of([(50, n)])
    f, scale = rs.freqs(rot, 1e4)
    t = dev(flat)
    x = t[:, 8:8 + heads * 256].unflatten(1, (heads, 256))
    apart = torch().empty((n, heads, 256), dtype=torch().int16, device="cuda")
    pkv.rope_rows(r, s, heads, x, apart)
    v = rs.bf16_values(flat[:, 8:8 + heads * 256].reshape(n, heads, 256))
    close(host(apart), *rs.turn(v, np.arange(41, 50), rot, pairs, f, scale))
    pkv.rope_rows(r, s, heads, x, x)
    got = host(t)
    assert np.array_equal(got[:, 8:8 + heads * 256].reshape(n, heads, 256), host(apart))
    assert np.array_equal(got[:, :8], flat[:, :8]) and np.array_equal(got[:, 8 + heads * 256:], flat[:, 8 + heads * 256:])


def test_infinities_and_nan_stay_in_their_pair():
    x = np.zeros((1, 1, 256), np.float32)
    x[0, 0, 3], x[0, 0, 40], x[0, 0, 200] = np.inf, np.nan, -np.inf
    out = torch().empty((1, 1, 256), dtype=torch().int16, device="cuda")
    pkv.rope_rows(pkv.rope(64, 1e4), seqs_of([(100, 1)]), 1, dev(rs.bf16_bits(x)), out)
    got = rs.bf16_values(host(out))[0, 0]
    bad = np.flatnonzero(~np.isfinite(got))
    assert set(bad) == {3, 35, 40 - 32, 40, 200} and got[200] == -np.inf


# ---- into the pages ------------------------------------------------------------------

class Pages:
    """Streams with their pages shuffled over one arena of NaN rows (ptok None: buffers of their own)."""

    def __init__(self, lay, lens, ptok, seed=0):
        t = torch()
        rng = np.random.default_rng(seed)
        self.lay, self.lens, self.ptok = lay, lens, ptok
        need = [-(-n // ptok) for n, _ in lens] if ptok else []
        self.n_pages = sum(need) + 3
        cap = ptok or max(4, -(-max(n for n, _ in lens) // 4) * 4)
        self.ps = pkv.page_elems(lay, cap)
        self.pos_page = cap
        ids = rng.permutation(self.n_pages).astype(np.int32)
        self.tables, at, self.seqs, self.keep = [], 0, [], []
        self.mem = t.full(((self.n_pages if ptok else len(lens)), self.ps), 0x7FC1, dtype=t.int16, device="cuda")
        for i, (n, m) in enumerate(lens):
            if ptok:
                self.tables.append(np.ascontiguousarray(ids[at:at + need[i]]))
                at += need[i]
                table = t.from_numpy(self.tables[-1]).cuda() if need[i] else t.zeros(1, dtype=t.int32, device="cuda")
                self.keep.append(table)
                g = pkv.pg(self.mem, table, self.ps, ptok, self.n_pages)
            else:
                self.tables.append(None)
                g = pkv.pg(self.mem[i], None, self.ps, cap)
            self.seqs.append(pkv.seq(g, n, m))

    def row(self, i, kind, head, pos, layer=0):
        """Offset of a row in the whole memory: 16-bit elements, bytes for e4m3."""
        at = pkv.pg_row(self.lay, self.seqs[i].pg, self.tables[i], layer, kind, head, pos)
        return at + (0 if self.ptok else i * self.ps * (2 if self.lay.kv_format == pkv.KV_E4M3 else 1))


@pytest.mark.parametrize("ptok", [4, 16, 20, 256, None])
@pytest.mark.parametrize("pairs,rot,hkv,hq,idx", [(HALF, 64, 2, 16, 128), (INTER, 256, 1, 4, 0), (HALF, 22, 3, 3, 128)])
def test_store_is_rows_then_store(ptok, pairs, rot, hkv, hq, idx):
    """bf16: the pages hold the bytes of rope_rows and store, and nothing else changed; the queries as by rope_rows."""
    rng = np.random.default_rng(5)
    lens = [(300, 5), (33, 33), (70, 0), (1, 1), (1030, 2)]
    lay = pkv.layout(3, hkv, 256, idx)
    a, b = Pages(lay, lens, ptok, 1), Pages(lay, lens, ptok, 1)
    n = sum(m for _, m in lens)
    q, k, v = (dev(rs.random_rows(rng, n, h, 256)) for h in (hq, hkv, hkv))
    ik = dev(rs.random_rows(rng, n, idx)) if idx else None
    r = pkv.rope(rot, 1e6, pairs, pkv.ROPE_LINEAR, factor=2.0)
    st = torch().zeros(1, dtype=torch().int32, device="cuda")
    q1, q2, k2 = torch().empty_like(q), torch().empty_like(q), torch().empty_like(k)
    pkv.rope_store(lay, a.seqs, 1, r, k, v, ik, n_q_heads=hq, q=q, q_out=q1, status=st)
    pkv.rope_rows(r, b.seqs, hkv, k, k2)
    pkv.rope_rows(r, b.seqs, hq, q, q2)
    pkv.store(lay, b.seqs, 1, k2, v, ik, status=st)
    assert torch().equal(a.mem, b.mem) and torch().equal(q1, q2) and int(st) == 0
    f, scale = rs.freqs(rot, 1e6, "linear", 2.0)
    close(host(q1), *rs.turn(rs.bf16_values(host(q)), places(lens), rot, pairs, f, scale))
    # and without the queries, out of one projection's rows
    flat = torch().cat([q.flatten(1), k.flatten(1), v.flatten(1)] + ([ik] if idx else []), 1)
    c = Pages(lay, lens, ptok, 1)
    parts = flat.split([hq * 256, hkv * 256, hkv * 256] + ([idx] if idx else []), 1)
    pkv.rope_store(lay, c.seqs, 1, r, parts[1].unflatten(1, (hkv, 256)), parts[2].unflatten(1, (hkv, 256)), parts[3] if idx else None)
    assert torch().equal(c.mem, b.mem)


@pytest.mark.parametrize("ptok", [4, 48, None])
@pytest.mark.parametrize("pairs,rot", [(HALF, 64), (INTER, 256), (HALF, 10)])
def test_e4m3_pages(ptok, pairs, rot):
    """Scales and codes of the rotated keys from float32; values as by store."""
    rng = np.random.default_rng(6)
    lens = [(130, 9), (64, 1)]
    lay = pkv.layout(2, 2, 256, 128, pkv.KV_E4M3)
    a, b = Pages(lay, lens, ptok, 2), Pages(lay, lens, ptok, 2)
    n = 10
    kb = rs.random_rows(rng, n, 2, 256)
    kb[3, 1] = 0                                          # a row of zeros
    k, v, ik = dev(kb), dev(rs.random_rows(rng, n, 2, 256)), dev(rs.random_rows(rng, n, 128))
    r = pkv.rope(rot, 1e4, pairs)
    pkv.rope_store(lay, a.seqs, 1, r, k, v, ik)
    pkv.store(lay, b.seqs, 1, k, v, ik)
    got, other = (m.mem.cpu().numpy().view(np.uint8).reshape(-1) for m in (a, b))
    f, scale = rs.freqs(rot, 1e4)
    want, size = rs.turn(rs.bf16_values(kb), places(lens), rot, pairs, f, scale)
    keys, at = np.zeros(got.shape, bool), 0
    for i, (length, m) in enumerate(lens):
        for p in range(length - m, length):
            for h in range(2):
                c0, s0 = a.row(i, pkv.K, h, p, 1), a.row(i, pkv.KS, h, p, 1)
                keys[c0:c0 + 256] = keys[s0:s0 + 4] = True
                s = got[s0:s0 + 4].view(np.float32)[0].astype(np.float64)
                w, e = want[at, h], rs.slack(size[at, h])
                # the scale: the largest value over 448, a division's rounding
                assert abs(s - np.abs(w).max() / 448) <= e.max() / 448 + 2.0 ** -24 * s
                x = orc.e4m3_to_double(got[c0:c0 + 256]) * s
                # a rounding to e4m3, 2^-10 of a unit for values below 2^-6 (a division's rounding beside it)
                assert (np.abs(x - w) <= np.maximum(2.0 ** -4 * np.abs(w), s * 2.0 ** -10) * (1 + 2.0 ** -20) + 2 * e).all()
            at += 1
    assert np.array_equal(got[~keys], other[~keys])


def test_given_positions_turn_the_rows_and_not_their_places():
    rng = np.random.default_rng(7)
    lay, lens = pkv.layout(1, 1, 256, 0), [(40, 4)]
    a, b = Pages(lay, lens, 16), Pages(lay, lens, 16)
    k, v = dev(rs.random_rows(rng, 4, 1, 256)), dev(rs.random_rows(rng, 4, 1, 256))
    pos = torch().tensor([7, -3, 100000, 2], dtype=torch().int32, device="cuda")
    k2 = torch().empty_like(k)
    r = pkv.rope(256)
    pkv.rope_store(lay, a.seqs, 0, r, k, v, pos=pos)
    pkv.rope_rows(r, b.seqs, 1, k, k2, pos=pos)
    pkv.store(lay, b.seqs, 0, k2, v)
    assert torch().equal(a.mem, b.mem)


def test_a_bad_page_is_reported_and_only_its_rows_left_out():
    t = torch()
    rng = np.random.default_rng(8)
    lay = pkv.layout(1, 2, 256, 128)
    for fmt in (pkv.KV_BF16, pkv.KV_E4M3):
        lay = pkv.layout(1, 2, 256, 128, fmt)
        ps = pkv.page_elems(lay, 16)
        mem = t.full((4, ps), 0x7FC1, dtype=t.int16, device="cuda")
        table = t.tensor([0, 9, 2], dtype=t.int32, device="cuda")
        st = t.zeros(1, dtype=t.int32, device="cuda")
        k, v, ik = dev(rs.random_rows(rng, 34, 2, 256)), dev(rs.random_rows(rng, 34, 2, 256)), dev(rs.random_rows(rng, 34, 128))
        pkv.rope_store(lay, [pkv.seq(pkv.pg(mem, table, ps, 16, 4), 34, 34)], 0, pkv.rope(64), k, v, ik, status=st)
        assert int(st) == pkv.DEV_BAD_PAGE
        assert (mem[1] == 0x7FC1).all() and (mem[3] == 0x7FC1).all() and not (mem[0] == 0x7FC1).all() and not (mem[2] == 0x7FC1).all()


def test_captured_on_another_stream_then_decoded():
    """A step as it is used: rope_store, then decode with the rotated queries, in a graph on a stream of its own, replayed on new rows."""
    t = torch()
    rng = np.random.default_rng(9)
    lay, length, hq = pkv.layout(1, 2, 256, 128), 200, 8
    a, b = Pages(lay, [(length, 1)], 16, 3), Pages(lay, [(length, 1)], 16, 3)
    r = pkv.rope(64, 1e6)
    k0, v0, ik0 = dev(rs.random_rows(rng, length, 2, 256)), dev(rs.random_rows(rng, length, 2, 256)), dev(rs.random_rows(rng, length, 128))
    for p in (a, b):
        pkv.store(lay, [pkv.seq(p.seqs[0].pg, length, length)], 0, k0, v0, ik0)
    q, k, v, ik = (t.empty(s, dtype=t.int16, device="cuda") for s in ((1, hq, 256), (1, 2, 256), (1, 2, 256), (1, 128)))
    q_out, out, ws = t.empty_like(q), t.empty_like(q), t.empty(max(64, pkv.decode_ws_size(lay, a.seqs, hq) // 4), device="cuda")

    def step(p):
        pkv.rope_store(lay, p.seqs, 0, r, k, v, ik, n_q_heads=hq, q=q, q_out=q_out)
        pkv.decode(lay, p.seqs, 0, hq, q_out, out, ws)

    side = t.cuda.Stream()
    t.cuda.synchronize()
    with t.cuda.stream(side):
        step(a)
        side.synchronize()
        g = t.cuda.CUDAGraph()
        with t.cuda.graph(g, stream=side):
            step(a)
        for seed in range(3):
            new = [dev(rs.random_rows(np.random.default_rng(seed), *x.shape)) for x in (q, k, v, ik)]
            for x, y in zip((q, k, v, ik), new):
                x.copy_(y)
            g.replay()
            got = out.clone()
            side.synchronize()
            q2, k2 = t.empty_like(q), t.empty_like(k)
            pkv.rope_rows(r, b.seqs, hq, q, q2)
            pkv.rope_rows(r, b.seqs, 2, k, k2)
            pkv.store(lay, b.seqs, 0, k2, v, ik)
            pkv.decode(lay, b.seqs, 0, hq, q2, out, ws)
            side.synchronize()
            assert t.equal(got, out)


@pytest.mark.parametrize("tokens,spare", [(1, 0), (3, 0), (3, 8), (2500, 0)])
def test_queries_turned_where_one_projection_has_them(tokens, spare):
    """q_out beside the keys, values and indexer rows of the same projection's rows: these go into the pages as ever."""
    rng, t = np.random.default_rng(tokens), torch()
    lay, lens = pkv.layout(1, 2, 256, 128), [(tokens + 50, tokens)]
    a, b = Pages(lay, lens, 16, 1), Pages(lay, lens, 16, 1)
    flat = dev(rs.random_rows(rng, tokens, 6 * 256 + 2 * 512 + 128 + spare))
    cut = lambda x: x[:, :6 * 256 + 2 * 512 + 128].split([6 * 256, 512, 512, 128], 1)  # noqa: E731
    parts, r = [x.contiguous() for x in cut(flat)], pkv.rope(64, 1e4)
    want, before = t.empty_like(parts[0]), flat.clone()
    pkv.rope_store(lay, b.seqs, 0, r, *parts[1:], n_q_heads=6, q=parts[0], q_out=want)
    q, k, v, ik = cut(flat)
    pkv.rope_store(lay, a.seqs, 0, r, k, v, ik, n_q_heads=6, q=q, q_out=q)
    assert t.equal(a.mem, b.mem) and t.equal(q, want) and t.equal(flat[:, 6 * 256:], before[:, 6 * 256:])
