"""What the windowed calls take from Python: tensors of the rows' types that hold
the launch's rows.  Stand-ins for device tensors: nothing runs on a GPU, and a
call that is let through ends in PKV_ECUDA where there is none."""
import pytest
import torch

from paged_kv_cache_pg_gb300 import build, pkv


class Device:
    """Looks like a contiguous tensor of device 0."""

    def __init__(self, shape, dtype=torch.bfloat16, at=0x100000):
        self._t, self._at = torch.empty(shape, dtype=dtype, device="meta"), at
        self.dtype, self.shape, self.nbytes, self.itemsize = dtype, self._t.shape, self._t.nbytes, self._t.itemsize

    def get_device(self):
        return 0

    def is_contiguous(self):
        return True

    def data_ptr(self):
        return self._at

    def numel(self):
        return self._t.numel()


@pytest.fixture(scope="module", autouse=True)
def lib():
    build.build()
    return pkv.load()


@pytest.fixture(autouse=True)
def device(monkeypatch):
    if torch.cuda.is_available():
        pytest.skip("stand-ins for device memory: only where no GPU could touch it")
    monkeypatch.setattr(pkv, "_current", (torch, lambda: 0, lambda dev: 0))


HQ, HKV, IDX = 8, 2, 128


def _call(which, n_new=(2, 1), **change):
    lay = pkv.layout(1, HKV, 256, IDX)
    g = pkv.Pg(0x100000, 0x200000, pkv.page_elems(lay, 16), 16, 64, 50, 0)
    seqs = [pkv.seq(g, 200 + i, n) for i, n in enumerate(n_new)]
    if change.pop("batch", False):
        seqs = pkv.batch(seqs)
    n = sum(n_new)
    a = dict(q=Device((n, HQ, 256)), out=Device((n, HQ, 256)), ws=Device((1 << 22,), torch.float32),
             status=Device((1,), torch.int32))
    if which == "decode":
        a.update(k_new=Device((n, HKV, 256)), v_new=Device((n, HKV, 256)), ik_new=Device((n, IDX)))
    a.update(change)
    f = pkv.window_decode if which == "decode" else pkv.window_prefill
    with pytest.raises(pkv.PkvError) as e:
        f(lay, seqs, 0, HQ, 100, 4, a.pop("q"), a.pop("out"), a.pop("ws"), stream=0, **a)
    return e.value.code


@pytest.mark.parametrize("which", ["decode", "prefill"])
@pytest.mark.parametrize("n_new", [(1,), (2, 1), (1, 0, 2, 3, 1, 1)])
@pytest.mark.parametrize("batch", [False, True])
def test_tensors_that_hold_the_launch_s_rows(which, n_new, batch):
    n, kw = sum(n_new), dict(n_new=n_new, batch=batch)
    assert _call(which, **kw) == pkv.ECUDA                                   # let through
    assert _call(which, q=Device((n, HQ, 256), torch.int16), out=Device((n + 3, HQ, 256), torch.uint16), **kw) == pkv.ECUDA
    assert _call(which, q=0x100000, out=0x100000, status=None, **kw) == pkv.ECUDA   # addresses are the caller's
    short = dict(q=(n, HQ, 255), out=(n, HQ - 1, 256))
    if which == "decode":
        short.update(k_new=(n, HKV, 255), v_new=(n - 1, HKV, 256), ik_new=(n, IDX - 1))
    for name, shape in short.items():
        assert _call(which, **{name: Device(shape)}, **kw) == pkv.EINVAL, name
        for dtype in (torch.float32, torch.float16, torch.int32, torch.uint8):
            assert _call(which, **{name: Device((n, HQ, 1024), dtype)}, **kw) == pkv.EINVAL, (name, dtype)
    for status in (Device((1,), torch.int64), Device((0,), torch.int32), Device((4,), torch.int8)):
        assert _call(which, status=status, **kw) == pkv.EINVAL
    assert _call(which, ws=0x100000, **kw) == pkv.EINVAL                     # an address says nothing of its size


def test_tables_have_to_be_tensors():
    with pytest.raises(pkv.PkvError) as e:
        pkv.tables_remap([0x100000], [1], [2], stream=0)
    assert e.value.code == pkv.EINVAL


@pytest.mark.parametrize("call", [pkv.window_decode, pkv.window_prefill])
def test_the_streams_have_to_be_streams(call):
    import ctypes
    with pytest.raises(pkv.PkvError) as e:
        call(pkv.layout(1, HKV, 256, IDX), (ctypes.c_int32 * 24)(), 0, HQ, 100, 4, 0x100000, 0x100000, None, stream=0)
    assert e.value.code == pkv.EINVAL


@pytest.mark.parametrize("big", [(1 << 32) + 5, 1 << 31, (1 << 40) + 1, -1])
def test_integers_beyond_32_bits_are_refused(big):
    lay = pkv.layout(1, HKV, 256, IDX)
    seqs = [pkv.seq(pkv.Pg(0x100000, 0x200000, pkv.page_elems(lay, 16), 16, 64, 50, 0), 200, 1)]
    arena = pkv.Arena(lay, 16, 0x200000, nbytes=2 * pkv.page_elems(lay, 16) * 4)
    rows = (0x100000, 0x100000, None)
    calls = [lambda: pkv.window_decode(lay, seqs, 0, HQ, big, 4, *rows, stream=0),
             lambda: pkv.window_decode(lay, seqs, 0, HQ, 100, big, *rows, stream=0),
             lambda: pkv.window_decode(lay, seqs, big, HQ, 100, 4, *rows, stream=0),
             lambda: pkv.window_decode(lay, seqs, 0, big, 100, 4, *rows, stream=0),
             lambda: pkv.window_prefill(lay, seqs, 0, HQ, big, 4, *rows, stream=0),
             lambda: pkv.window_prefill(lay, seqs, 0, HQ, 100, big, *rows, stream=0),
             lambda: pkv.window_decode_ws_size(lay, seqs, HQ, big, 4),
             lambda: pkv.window_prefill_ws_size(lay, seqs, HQ, 100, big),
             lambda: pkv.window_dead_pages(16, 200, big, 4), lambda: pkv.window_dead_pages(16, big, 100, 4),
             lambda: pkv.pages_copy(lay, 16, 0x200000, big, [0], [1], stream=0),
             lambda: pkv.pages_copy(lay, big, 0x200000, 4, [0], [1], stream=0),
             lambda: arena.fork([], big), lambda: arena.compact(big)]
    for i, call in enumerate(calls):
        with pytest.raises(pkv.PkvError) as e:
            call()
        assert e.value.code == pkv.EINVAL, i
    arena.close()
