"""Ropes and their calls' checks, without a GPU: frequencies against the formulas, refused arguments."""
import ctypes
import math

import numpy as np
import pytest

from paged_kv_cache_pg_gb300 import build, pkv

import rope_setup as rs


@pytest.fixture(scope="module", autouse=True)
def lib():
    build.build()
    return pkv.load()


KINDS = {"plain": pkv.ROPE_PLAIN, "linear": pkv.ROPE_LINEAR, "ntk": pkv.ROPE_NTK, "yarn": pkv.ROPE_YARN,
         "bands": pkv.ROPE_BANDS}


@pytest.mark.parametrize("kind", list(KINDS))
@pytest.mark.parametrize("rot,base,factor,original", [(64, 1e6, 4.0, 8192), (256, 1e4, 8.0, 4096), (4, 5e5, 1.0, 32768),
                                                     (250, 1e4, 2.5, 100)])
def test_frequencies(kind, rot, base, factor, original):
    r = pkv.rope(rot, base, pkv.ROPE_HALF, KINDS[kind], factor=factor, original=original)
    f, scale = rs.freqs(rot, base, kind, factor, original)
    got = np.array([int(t) for t in r.turns[:rot // 2]], dtype=np.float64) / 2.0 ** 64 * 2 * math.pi
    # a few roundings of pow, of the ramp and of the division by a turn in 64 bits; the whole
    # number of 2^-64 of a turn that is kept is up to one off: 2 pi 2^-64 of a radian
    assert np.allclose(got, f % (2 * math.pi), rtol=1e-13, atol=2 * math.pi * 2.0 ** -64)
    assert abs(r.scale - scale) <= 2.0 ** -24 * scale
    assert r.rot_dim == rot and r.pairs == pkv.ROPE_HALF and r.reserved == 0
    assert all(t == 0 for t in r.turns[rot // 2:])


def test_own_bounds_and_scale():
    r = pkv.rope(128, 1e4, pkv.ROPE_INTERLEAVED, pkv.ROPE_YARN, factor=16.0, original=4096, fast=16, slow=2, scale=0.5)
    f, _ = rs.freqs(128, 1e4, "yarn", 16.0, 4096, 16, 2)
    got = np.array([int(t) for t in r.turns[:64]], dtype=np.float64) / 2.0 ** 64 * 2 * math.pi
    assert np.allclose(got, f, rtol=1e-13, atol=2 * math.pi * 2.0 ** -64) and r.scale == 0.5


def test_frequencies_of_the_callers_own():
    f = [1.0, -0.25, 7.5, 0.0, 1e-9]
    r = pkv.rope_from_freqs(f, pkv.ROPE_INTERLEAVED, 2.0)
    want = [(x / (2 * math.pi)) % 1.0 for x in f]
    got = [int(t) / 2.0 ** 64 for t in r.turns[:5]]
    assert np.allclose(got, want, rtol=1e-13, atol=1e-18) and r.rot_dim == 10 and r.scale == 2.0
    with pytest.raises(pkv.PkvError):
        pkv.rope_from_freqs([float("nan")])
    with pytest.raises(pkv.PkvError):
        pkv.rope_from_freqs([1.0] * 129)
    with pytest.raises(pkv.PkvError):
        pkv.rope_from_freqs([])
    # a negative frequency of less than the smallest fraction is no turn at all
    assert int(pkv.rope_from_freqs([-1e-300]).turns[0]) in (0, 2 ** 64 - 1, 2 ** 64 - 2 ** 11)


@pytest.mark.parametrize("bad", [dict(rot_dim=0), dict(rot_dim=3), dict(rot_dim=258), dict(base=1.0), dict(base=float("nan")),
                                 dict(base=float("inf")), dict(pairs=2), dict(scaling=5), dict(scaling=pkv.ROPE_LINEAR, factor=0.5),
                                 dict(scaling=pkv.ROPE_NTK, rot_dim=2, factor=2.0), dict(scaling=pkv.ROPE_YARN, factor=2.0, original=0),
                                 dict(scaling=pkv.ROPE_BANDS, factor=2.0, original=100, fast=1.0, slow=1.0),
                                 dict(scaling=pkv.ROPE_BANDS, factor=2.0, original=100, fast=4.0, slow=-1.0),
                                 dict(scaling=pkv.ROPE_NTK, rot_dim=4, base=1e300, factor=1e200), dict(scale=float("inf")),
                                 dict(rot_dim=-2), dict(rot_dim=2 ** 32 + 64)])
def test_refused_ropes(bad):
    with pytest.raises(pkv.PkvError) as e:
        pkv.rope(**{**dict(rot_dim=64), **bad})
    assert e.value.code == pkv.EINVAL


# ---- the calls' checks (nothing is launched) -------------------------------------

def _rows(lib, seqs=((10, 2),), rope=None, n_heads=4, dim=256, x=0x10000, xs=0, out=0x900000, os_=0, pos=None):
    arr = (pkv.Seq * max(1, len(seqs)))(*[pkv.seq(pkv.Pg(), n, m) for n, m in seqs])
    r = rope if rope is not None else pkv.rope(64)
    return lib.pkv_rope_rows(ctypes.addressof(r), ctypes.addressof(arr), len(seqs), pos, n_heads, dim, x, xs, out, os_, None)


def test_rows_refuses(lib):
    assert _rows(lib, seqs=()) == pkv.OK                 # nothing to do
    assert _rows(lib, seqs=((10, 0),)) == pkv.OK
    for bad in (dict(dim=64), dict(dim=0), dict(n_heads=0), dict(n_heads=1 << 20), dict(seqs=((1, 2),)), dict(seqs=((-1, 0),)),
                dict(seqs=((5, -1),)), dict(x=None), dict(out=None), dict(x=0x10008), dict(out=0x900002), dict(xs=1020), dict(xs=1028),
                dict(os_=4 * 256 - 8), dict(rope=pkv.rope(256), dim=128), dict(seqs=((1 << 30, 1 << 30), (1 << 30, 1 << 30))),
                dict(out=0x10000 + 512),                 # in the middle of its own input
                dict(out=0x10000, os_=2048),             # in place with another stride
                dict(out=0x10000 + 2048, xs=1024, os_=1024)):
        assert _rows(lib, **bad) == pkv.EINVAL, bad
    bad_rope = pkv.rope(64)
    bad_rope.rot_dim = 7
    assert _rows(lib, rope=bad_rope) == pkv.EINVAL
    assert lib.pkv_rope_rows(None, None, 0, None, 4, 256, None, 0, None, 0, None) == pkv.EINVAL


def _store(lib, fmt=pkv.KV_BF16, idx=128, rope=True, layer=0, nq=4, q=0x100000, qs=0, qo=0x200000, qos=0, k=0x300000, ks=0, v=0x400000,
           vs=0, ik=0x500000, iks=0, length=10, n_new=2, n_table=4):
    lay = pkv.layout(2, 2, 256, idx, fmt)
    s = pkv.seq(pkv.Pg(0x1000000, 0x2000000, pkv.page_elems(lay, 16), 16, 8, n_table, 0), length, n_new)
    r = pkv.rope(64)
    return lib.pkv_rope_store(ctypes.addressof(lay), ctypes.addressof(s), 1, layer, ctypes.addressof(r) if rope else None, None, nq, q, qs, qo, qos, k, ks, v, vs, ik, iks,
                              None, None)


def test_store_refuses(lib):
    assert _store(lib, n_new=0) == pkv.OK
    for bad in (dict(rope=False), dict(layer=2), dict(nq=0), dict(q=0x100004), dict(qo=None), dict(qo=0x100000 + 512), dict(qs=512),
                dict(ks=256), dict(ks=516), dict(vs=260), dict(k=None), dict(v=None), dict(k=0x300008), dict(ik=None), dict(ik=0x500004),
                dict(iks=64), dict(length=65), dict(n_new=11), dict(n_new=-1)):
        assert _store(lib, **bad) == pkv.EINVAL, bad
    # the strides of rows that are not there do not count
    assert _store(lib, q=None, qs=4, n_new=0) == pkv.OK


@pytest.mark.parametrize("n_new", [1, 2])
@pytest.mark.parametrize("bad", [
    dict(qo=0x300000), dict(qo=0x300000 + 512), dict(qo=0x400000 - 1024), dict(qo=0x500000 - 2048 + 16), dict(qo=0x500000 + 128),
    dict(qo=0x400000, q=0x400000),                                                         # the queries and the values are the same rows
    # one projection's rows of 2,304 elements (1,024 of queries, 2 heads of keys, 64 unused, 2 of values, 128 indexer elements, 64 unused):
    # queries out over the keys, the values' first elements and the indexer's last ones
    *(dict(q=0x700000, qos=2304, k=0x100000 + 2048, ks=2304, v=0x100000 + 3200, vs=2304, ik=0x100000 + 4224, iks=2304, qo=0x100000 + at)
      for at in (2048, 3200 - 2048 + 16, 4224 + 240))])
def test_store_refuses_queries_written_over_its_other_rows(lib, bad, n_new):
    assert _store(lib, n_new=n_new, **bad) == pkv.EINVAL


def test_python_refuses_what_ctypes_would_cut():
    lay = pkv.layout(1, 2)
    for call in (lambda: pkv.rope_store(lay, [], 1 << 32, pkv.rope(64), None, None),
                 lambda: pkv.rope_store(lay, [], 0, pkv.rope(64), None, None, n_q_heads=-1),
                 lambda: pkv.rope_store(lay, [], 0, None, None, None),
                 lambda: pkv.rope_rows(pkv.rope(64), [], 1 << 33, 0, 0),
                 lambda: pkv.rope_rows(None, [], 1, 0, 0)):
        with pytest.raises(pkv.PkvError) as e:
            call()
        assert e.value.code == pkv.EINVAL


def test_rows_that_lie_apart():
    """Slices of wider rows are taken with their stride; what does not lie together, is too short or is one row expanded is refused."""
    torch = pytest.importorskip("torch")
    rows = lambda t, tokens, width: pkv._token_rows("x", "x", t, -1, tokens, width)  # noqa: E731
    wide = torch.zeros((6, 40, 8), dtype=torch.int16)
    part = wide[:, 3:19]
    assert rows(part, 6, 128) == (part.data_ptr(), 320) and rows(part, 4, 128) == (part.data_ptr(), 320)
    assert rows(part.flatten(1), 6, 128) == (part.data_ptr(), 320)      # (still a view)
    assert rows(wide[::2, :16], 3, 128) == (wide.data_ptr(), 640) and rows(wide, 6, 320) == (wide.data_ptr(), 0)
    one = torch.zeros((4, 8), dtype=torch.int16)
    assert rows(one.expand(5, 4, 8), 1, 32) == (one.data_ptr(), 0)
    assert rows(wide[:1, 3:19], 1, 128)[1] == 0 and rows(wide[:0, 3:19], 0, 128)[1] == 0
    for bad, tokens, width in ((one.expand(5, 4, 8), 5, 32), (part, 7, 128), (part, 6, 120), (wide[:, ::2], 6, 160), (wide[..., :4], 6, 160),
                               (wide.transpose(0, 1), 6, 48), (part.float(), 6, 128), (torch.zeros(40, dtype=torch.int16)[::2], 4, 5)):
        with pytest.raises(pkv.PkvError):
            rows(bad, tokens, width)


def test_contiguous_rows_of_another_width():
    """A longer contiguous tensor is packed rows where its shape says so; wider or narrower tokens are refused, as their slices are."""
    torch = pytest.importorskip("torch")
    rows = lambda t, tokens, width: pkv._token_rows("x", "x", t, -1, tokens, width)  # noqa: E731
    z = lambda *shape: torch.zeros(shape, dtype=torch.int16)  # noqa: E731
    for good, tokens, width in ((z(9, 16, 256), 6, 4096), (z(9, 4096), 6, 4096), (z(2, 3, 16, 256), 6, 4096), (z(3, 3, 16, 256), 6, 4096),
                                (z(1, 9, 16, 256), 6, 4096), (z(9, 1, 256), 6, 256), (z(9 * 16, 256), 6, 4096), (z(9 * 4096), 6, 4096),
                                (z(9, 128), 6, 128), (z(9 * 4, 128), 6, 512), (z(9, 16, 256), 1, 2048), (z(9, 16, 256), 0, 2048),
                                (z(9, 128), 6, 0), (z(12, 8, 256), 6, 4096), (z(8, 16, 256)[:6], 6, 4096)):
        assert rows(good, tokens, width) == (good.data_ptr(), 0), (good.shape, tokens, width)
    for bad, tokens, width in ((z(6, 16, 256), 6, 2048), (z(9, 4096), 6, 2048), (z(13, 8, 256), 6, 4096), (z(9, 3, 128), 6, 256), (z(9, 2, 128), 4, 512),
                               (z(6, 4096 + 8), 6, 4096), (z(6, 2, 16, 256), 6, 2048), (z(6, 256), 6, 128 * 3)):
        with pytest.raises(pkv.PkvError):
            rows(bad, tokens, width)
    # as it is called: queries of 16 heads told to be of 8, 6 tokens
    pkv_rows = lambda heads: pkv._token_rows("pkv_rope_rows", "x", z(6, 16, 256), -1, 6, heads * 256)  # noqa: E731
    assert pkv_rows(16)[1] == 0
    with pytest.raises(pkv.PkvError):
        pkv_rows(8)
