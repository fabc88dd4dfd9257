"""Sharing and compaction of the page arena, and the refusals of the page
copies and the table rewrite: no GPU needed."""
import ctypes

import numpy as np
import pytest

from paged_kv_cache_pg_gb300 import build, pkv


@pytest.fixture(scope="module", autouse=True)
def lib():
    build.build()
    return pkv.load()


def _arena(n_pages, ptok=16):
    lay = pkv.layout(1, 1, 256, 0)
    return pkv.Arena(lay, ptok, 0x200000, nbytes=2 * pkv.page_elems(lay, ptok) * n_pages)


def _code(f, *a, **k):
    with pytest.raises(pkv.PkvError) as e:
        f(*a, **k)
    return e.value.code


@pytest.fixture()
def arena():
    a = _arena(12)
    yield a
    a.close()


class Events:
    """Fake event operations: releases wait until `done` is set."""

    def __init__(self):
        self.done = False
        E = pkv.EventOps

        def record(ctx, stream, ev):
            ev[0] = 1
            return 0
        self.ops = E(E.RECORD(record), E.QUERY(lambda ctx, ev: 0 if self.done else 1),
                     E.DESTROY(lambda ctx, ev: None), None)


def test_fork_shares_whole_pages_and_gives_a_fresh_tail(arena):
    ids = arena.take(3)
    out, copy = arena.fork(ids, 40)                      # 16 + 16 + 8 positions
    assert out.tolist() == [0, 1, 3] and copy == (2, 3, 8)
    assert arena.holders([0, 1, 2, 3, 4]).tolist() == [2, 2, 1, 1, 0]
    assert arena.info()[1] == 8
    arena.give(ids, defer=False)                         # the first stream ends
    assert arena.holders([0, 1, 2, 3]).tolist() == [1, 1, 0, 1]
    assert arena.info()[1] == 9
    arena.give(out, defer=False)
    assert arena.info()[1] == 12


def test_fork_of_whole_pages_copies_nothing(arena):
    ids = arena.take(2)
    out, copy = arena.fork(ids, 32)
    assert out.tolist() == [0, 1] and copy is None and arena.info()[1] == 10
    assert arena.fork([], 0)[0].size == 0
    # a fork of the fork
    again, copy = arena.fork(out, 32)
    assert arena.holders([0, 1]).tolist() == [3, 3]


def test_fork_keeps_pages_behind_a_window_as_gone(arena):
    ids = arena.take(4)
    arena.give([ids[1]], defer=False)
    ids[1] = -1
    out, copy = arena.fork(ids, 64)
    assert out.tolist() == [0, -1, 2, 3] and copy is None


def test_fork_refusals_change_nothing(arena):
    ids = arena.take(12)
    assert _code(arena.fork, ids[:2], 20) == pkv.EAGAIN          # no page for the tail
    assert arena.holders(ids).tolist() == [1] * 12
    arena.give(ids[4:], defer=False)
    for bad, n in [([0], 17), ([0, 1], 16), ([0, 0], 32), ([0, 4], 32), ([0, 12], 32), ([-2, 0], 32), ([0, -1], 20)]:
        assert _code(arena.fork, bad, n) == pkv.EINVAL, (bad, n)
    run = arena.run_take(1)
    assert _code(arena.fork, [run], 16) == pkv.EINVAL
    assert arena.holders([run]).tolist() == [0]
    assert arena.holders(range(4)).tolist() == [1] * 4
    assert _code(arena.holders, [12]) == pkv.EINVAL
    assert _code(arena.holders, [-1]) == pkv.EINVAL


def test_a_shared_page_takes_as_many_gives_as_holders(arena):
    ev = Events()
    arena.set_event_ops(ev.ops)
    ids = arena.take(1)
    arena.fork(ids, 16)
    arena.give(ids, stream=1)
    assert arena.holders(ids).tolist() == [1] and arena.info()[1] == 11
    arena.give(ids, stream=1)
    assert arena.holders(ids).tolist() == [0] and arena.info()[1] == 11
    assert _code(arena.give, ids, stream=1) == pkv.EINVAL
    assert _code(arena.fork, ids, 16) == pkv.EINVAL       # every holder has given it
    ev.done = True
    assert arena.info()[1] == 12


def test_compact_moves_the_highest_pages_to_the_lowest_holes(arena):
    arena.take(10)
    arena.give([1, 4, 5], defer=False)                   # held: 0 2 3 6 7 8 9
    src, dst = arena.compact(2)
    assert src.tolist() == [9, 8] and dst.tolist() == [1, 4]
    assert arena.info()[1] == 3                          # 5, 10, 11: src is held until given
    arena.give(src, defer=False)
    src, dst = arena.compact(100)
    assert src.tolist() == [7] and dst.tolist() == [5]
    arena.give(src, defer=False)
    assert arena.info()[1] == 5
    assert arena.compact(100)[0].size == 0
    assert arena.holders(range(12)).tolist() == [1] * 7 + [0] * 5


def test_compact_makes_room_for_a_run(arena):
    arena.take(12)
    arena.give([0, 3, 6, 9], defer=False)
    assert _code(arena.run_take, 2) == pkv.EAGAIN
    src, dst = arena.compact(100)
    assert src.tolist() == [11, 10, 8] and dst.tolist() == [0, 3, 6]
    arena.give(src, defer=False)
    assert arena.run_take(3) == 9                        # 9, 10, 11


def test_compact_moves_holders_and_leaves_runs_and_going_pages(arena):
    ev = Events()
    arena.set_event_ops(ev.ops)
    ids = arena.take(9)
    run = arena.run_take(2)                              # 10, 11
    arena.fork([8], 16)                                  # page 8: two holders
    arena.fork([7], 16)
    arena.give([7], stream=1)                            # page 7: two holders, one going
    arena.give([6], stream=1)                            # page 6: going
    arena.give([0, 2], stream=1)
    ev.done = True
    assert arena.info()[1] == 4                          # 0 2 6 9
    ev.done = False
    arena.fork([7], 16)
    arena.give([7], stream=1)                            # again two holders, one going
    src, dst = arena.compact(100)
    assert src.tolist() == [8, 7] and dst.tolist() == [0, 2]
    assert arena.holders([0, 2, 8, 7]).tolist() == [2, 1, 1, 1]
    arena.give(src, stream=1)
    assert arena.holders([8, 7]).tolist() == [0, 0] and arena.info()[1] == 2
    ev.done = True
    assert arena.info()[1] == 4
    assert arena.run_map(run, 2, [16])                   # the run is where it was


def test_books_follow_a_model_over_random_forks_gives_and_compactions():
    rng = np.random.default_rng(3)
    for trial in range(4):
        n = int(rng.integers(6, 40))
        a = _arena(n)
        streams, holders = [], np.zeros(n, int)
        for _ in range(300):
            op = rng.integers(0, 4)
            if op == 0:
                k = int(rng.integers(1, 5))
                free = np.flatnonzero(holders == 0)
                if free.size < k:
                    assert _code(a.take, k) == pkv.EAGAIN
                else:
                    ids = a.take(k)
                    assert ids.tolist() == free[:k].tolist()
                    holders[ids] += 1
                    streams.append(ids.copy())
            elif op == 1 and streams:
                ids = streams[int(rng.integers(len(streams)))]
                length = int(rng.integers(16 * ids.size - 15, 16 * ids.size + 1))
                free = np.flatnonzero(holders == 0)
                if length % 16 and free.size == 0:
                    assert _code(a.fork, ids, length) == pkv.EAGAIN
                else:
                    out, copy = a.fork(ids, length)
                    want = ids.copy()
                    if length % 16:
                        assert copy == (ids[-1], free[0], length % 16)
                        want[-1] = free[0]
                    else:
                        assert copy is None
                    assert out.tolist() == want.tolist()
                    holders[out] += 1
                    streams.append(out.copy())
            elif op == 2 and streams:
                ids = streams.pop(int(rng.integers(len(streams))))
                a.give(ids, defer=False)
                holders[ids] -= 1
            elif op == 3:
                most = int(rng.integers(0, 6))
                src, dst = a.compact(most)
                held, free = np.flatnonzero(holders)[::-1], np.flatnonzero(holders == 0)
                k = min(most, held.size, free.size)
                pairs = [(s, d) for s, d in zip(held[:k], free[:k]) if d < s]
                assert [(int(s), int(d)) for s, d in zip(src, dst)] == pairs
                to = np.arange(n)
                to[src] = dst
                streams = [to[s] for s in streams]
                holders[dst], holders[src] = holders[src], 0
                a.give(src, defer=False)
            assert a.holders(range(n)).tolist() == holders.tolist()
            assert a.info()[1] == int((holders == 0).sum())
        a.close()


# ---- refusals before any launch ----------------------------------------------------

def _copy(src, dst, n_pos=None, lay=None, ptok=16, base=0x10000, n_pages=8):
    lay = lay or pkv.layout(2, 2)
    a = [np.ascontiguousarray(x, np.int32) if x is not None else None for x in (src, dst, n_pos)]
    p = [x.ctypes.data if x is not None else None for x in a]
    return pkv.load().pkv_pages_copy(ctypes.byref(lay), ptok, base, n_pages, *p, len(src), None)


def test_copy_refusals():
    assert _copy([0], [8]) == pkv.EINVAL                 # outside the arena
    assert _copy([-1], [0]) == pkv.EINVAL
    assert _copy([0, 1], [2, 2]) == pkv.EINVAL           # a page written twice
    assert _copy([0, 1], [1, 2]) == pkv.EINVAL           # written and read
    assert _copy([3], [3]) == pkv.EINVAL
    assert _copy([0], [1], [17]) == pkv.EINVAL
    assert _copy([0], [1], [-1]) == pkv.EINVAL
    assert _copy([0], [1], base=0x10008) == pkv.EINVAL
    assert _copy([0], [1], base=None) == pkv.EINVAL
    assert _copy([0], [1], ptok=18) == pkv.EINVAL
    assert _copy([0], [1], n_pages=0) == pkv.EINVAL
    assert _copy([0], [1], lay=pkv.layout(1, 64), ptok=1 << 20) == pkv.EINVAL   # a layer over 32 GB
    assert _copy([0], [1], lay=pkv.layout(0, 2)) == pkv.EINVAL
    assert _copy([], []) == pkv.OK                       # nothing to do, nothing launched
    assert _copy([0, 2], [1, 3], [0, 0]) == pkv.OK
    lay = pkv.layout(2, 2)
    f = pkv.load().pkv_pages_copy
    one = np.zeros(1, np.int32).ctypes.data
    assert f(ctypes.byref(lay), 16, 0x10000, 8, None, one, None, 1, None) == pkv.EINVAL
    assert f(ctypes.byref(lay), 16, 0x10000, 8, one, one, None, -1, None) == pkv.EINVAL
    assert _code(pkv.pages_copy, lay, 16, 0x10000, 8, [0, 1], [2], stream=0) == pkv.EINVAL
    assert _code(pkv.pages_copy, lay, 16, 0x10000, 8, [0], [2], n_pos=[1, 1], stream=0) == pkv.EINVAL


def _remap(tables, sizes, src, dst):
    t = (ctypes.c_void_p * max(1, len(tables)))(*tables)
    n = (ctypes.c_int32 * max(1, len(sizes)))(*sizes)
    s, d = (np.ascontiguousarray(x, np.int32) for x in (src, dst))
    return pkv.load().pkv_tables_remap(t, n, len(tables), s.ctypes.data, d.ctypes.data, len(src), None)


def test_remap_refusals():
    ok = 0x10000
    assert _remap([ok], [4], [1, 1], [2, 3]) == pkv.EINVAL
    assert _remap([ok], [4], [1, 2], [3, 3]) == pkv.EINVAL
    assert _remap([ok], [4], [1, 2], [2, 3]) == pkv.EINVAL
    assert _remap([ok], [4], [-1], [2]) == pkv.EINVAL
    assert _remap([ok], [4], [1], [-2]) == pkv.EINVAL
    assert _remap([ok], [-1], [1], [2]) == pkv.EINVAL
    assert _remap([None], [4], [1], [2]) == pkv.EINVAL
    assert _remap([ok + 2], [4], [1], [2]) == pkv.EINVAL
    assert _remap([], [], [1], [2]) == pkv.OK            # nothing to rewrite
    assert _remap([None], [0], [1], [2]) == pkv.OK
    assert _remap([ok], [4], [], []) == pkv.OK
    f = pkv.load().pkv_tables_remap
    assert f(None, None, 1, None, None, 0, None) == pkv.EINVAL
    assert f(None, None, 0, None, None, 1, None) == pkv.EINVAL
    assert f(None, None, -1, None, None, 0, None) == pkv.EINVAL
    assert _code(pkv.tables_remap, [], [1], [2, 3], stream=0) == pkv.EINVAL


def test_calls_take_only_contiguous_tensors_of_the_device():
    import torch
    lay = pkv.layout(1, 1, 256, 0)
    assert _code(pkv.pages_copy, lay, 16, torch.zeros(1 << 16, dtype=torch.int16), 2, [0], [1], stream=0) == pkv.EINVAL
    assert _code(pkv.tables_remap, [torch.zeros(4, dtype=torch.int32)], [0], [1], stream=0) == pkv.EINVAL


@pytest.mark.parametrize("bad", [[1 << 32], np.array([5 + (1 << 32)]), [1.5], [float("nan")], [-(1 << 31) - 1]])
def test_lists_of_other_than_32_bit_integers_are_refused(bad):
    lay = pkv.layout(1, 1, 256, 0)
    for call in (lambda: pkv.pages_copy(lay, 16, 0x1000, 8, bad, [1], stream=0),
                 lambda: pkv.pages_copy(lay, 16, 0x1000, 8, [1], [2], n_pos=bad, stream=0),
                 lambda: pkv.tables_remap([], bad, [1], stream=0)):
        with pytest.raises(pkv.PkvError) as e:
            call()
        assert e.value.code == pkv.EINVAL
