"""Checks of the calls over shared pages, without a GPU: refused arguments (nothing is launched)."""
import ctypes

import pytest

from paged_kv_cache_pg_gb300 import build, pkv


@pytest.fixture(scope="module", autouse=True)
def lib():
    build.build()
    return pkv.load()


PTOK = 16


def _call(lib, seqs=((100, 1, 0), (90, 2, 0)), groups=((2, 3),), fmt=pkv.KV_BF16, layer=0, hq=4, q=0x100000, k=None, v=None, ik=None,
          out=0x200000, ws=0x300000, ws_bytes=1 << 30, change=None, size=False, hkv=2, idx=128):
    """seqs: (len, n_new, 1 for a contiguous stream); change(pg descriptors)."""
    lay = pkv.layout(2, hkv, 256, idx, fmt)
    ps = pkv.page_elems(lay, PTOK)
    pgs = []
    for n, _, contiguous in seqs:
        cap = max(4, -(-n // 4) * 4)
        pgs.append(pkv.Pg(0x1000000, None, pkv.page_elems(lay, cap), cap, 1, 1, 0) if contiguous
                   else pkv.Pg(0x1000000, 0x2000000, ps, PTOK, 500, 50, 0))
    if change:
        change(pgs)
    arr = (pkv.Seq * max(1, len(seqs)))(*[pkv.seq(g, n, m) for g, (n, m, _) in zip(pgs, seqs)])
    gr = (pkv.Group * max(1, len(groups)))(*[pkv.Group(*g) for g in groups])
    if size:
        out = ctypes.c_size_t()
        return lib.pkv_prefix_decode_ws_size(ctypes.byref(lay), arr, len(seqs), ctypes.addressof(gr), len(groups), hq, ctypes.byref(out))
    return lib.pkv_prefix_decode(ctypes.addressof(lay), ctypes.addressof(arr), len(seqs), ctypes.addressof(gr), len(groups), layer, hq, q, k, v,
                                 ik, out, ws, ws_bytes, None, None)


def _other(**fields):
    def change(pgs):
        for name, value in fields.items():
            setattr(pgs[1], name, value)
    return change


SHORT = pkv.page_elems(pkv.layout(2, 2, 256, 128), 32)


@pytest.mark.parametrize("bad", [
    dict(groups=()), dict(groups=((1, 3),)), dict(groups=((3, 3),)), dict(groups=((2, 3), (1, 0))), dict(groups=((0, 3), (2, 3))),
    dict(groups=((-1, 3), (3, 3))), dict(groups=((2, -1),)), dict(groups=((1, 0), (1, 0), (1, 0))),
    dict(groups=((2, 6),)),                                         # past the second stream's cached rows (90 - 2)
    dict(groups=((2, 51),), seqs=((5000, 1, 0), (5000, 1, 0))),     # past a table's end, and the length past it
    dict(seqs=((100, 1, 0), (90, 2, 1))), dict(seqs=((100, 1, 1), (100, 1, 1))),
    dict(change=_other(base=0x4000000)), dict(change=_other(n_pages=400)), dict(change=_other(page_pos=32, page_elems=SHORT)),
    dict(change=_other(n_table=2)), dict(seqs=((100, 17, 0), (90, 2, 0))), dict(hq=3), dict(hq=0), dict(layer=2), dict(layer=-1),
    dict(seqs=(((1 << 29) + 4, 1, 1),), groups=((1, 0),)),
    dict(seqs=((10, 11, 0), (90, 2, 0)), groups=((2, 0),)), dict(seqs=tuple((100, 1, 0) for _ in range(65)), groups=((65, 1),))])
@pytest.mark.parametrize("size", [False, True])
def test_refuses(lib, bad, size):
    if size and "layer" in bad:
        return
    assert _call(lib, size=size, **bad) == pkv.EINVAL


def test_nothing_to_do(lib):
    """Streams without new tokens, and no streams: fine without a GPU where no kernel runs."""
    rc = _call(lib, seqs=((100, 0, 0), (90, 0, 0)), q=None, out=None, ws=None, ws_bytes=0)
    assert rc in (pkv.OK, pkv.ECUDA)   # (ECUDA: no GPU to ask for its size)


def test_python_refuses():
    lay = pkv.layout(1, 2)
    g = pkv.Pg(0x1000000, 0x2000000, pkv.page_elems(lay, PTOK), PTOK, 500, 50, 0)
    seqs = [pkv.seq(g, 100, 1), pkv.seq(g, 90, 1)]
    for groups in ([(2, -3)], [(1 << 32, 0)], [(2, 1 << 31)], (pkv.Seq * 1)(), [(1, 0)], []):
        with pytest.raises(pkv.PkvError) as e:
            pkv.prefix_decode_ws_size(lay, seqs, groups, 4)
        assert e.value.code == pkv.EINVAL


def test_nothing_to_do_needs_no_gpu(lib):
    """A call without new tokens, or without streams, returns before it asks for a GPU."""
    assert _call(lib, seqs=((100, 0, 0), (90, 0, 0)), q=None, out=None, ws=None, ws_bytes=0) == pkv.OK
    assert _call(lib, seqs=(), groups=(), q=None, out=None, ws=None, ws_bytes=0) == pkv.OK
