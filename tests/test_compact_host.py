"""Compactions planned one after another before the vacated pages are given
back: no GPU needed."""
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


def test_a_page_that_a_plan_has_vacated_is_not_moved_again():
    a = _arena(12)
    a.take(10)
    a.give([1, 4, 5], defer=False)                       # held: 0 2 3 6 7 8 9
    first = a.compact(1)
    second = a.compact(1)
    assert [x.tolist() for x in first + second] == [[9], [1], [8], [4]]
    third = a.compact(100)
    assert [x.tolist() for x in third] == [[7], [5]]
    assert a.holders([9, 8, 7]).tolist() == [1, 1, 1]    # the caller's, until given
    assert a.compact(100)[0].size == 0
    a.give([9, 8, 7], defer=False)
    assert a.holders(range(12)).tolist() == [1] * 7 + [0] * 5 and a.info()[1] == 5
    # taken anew, they are pages like others
    assert a.take(3).tolist() == [7, 8, 9]
    a.give([0], defer=False)
    assert [x.tolist() for x in a.compact(5)] == [[9], [0]]
    a.close()


def test_plans_in_a_row_follow_a_model():
    rng = np.random.default_rng(11)
    for trial in range(6):
        n = int(rng.integers(8, 40))
        a = _arena(n)
        held, owed = np.zeros(n, bool), []               # owed: vacated, not yet given
        for _ in range(200):
            op = int(rng.integers(0, 4))
            if op == 0:
                free = np.flatnonzero(~held)
                k = int(rng.integers(0, free.size + 1))
                assert a.take(k).tolist() == free[:k].tolist()
                held[free[:k]] = True
            elif op == 1:
                live = [p for p in np.flatnonzero(held) if p not in owed]
                ids = rng.permutation(np.array(live, np.int32))[:int(rng.integers(0, len(live) + 1))]
                a.give(ids, defer=False)
                held[ids] = False
            elif op == 2:
                most = int(rng.integers(0, 5))
                src, dst = a.compact(most)
                want, free = [], np.flatnonzero(~held)
                for p in np.flatnonzero(held)[::-1]:
                    if p not in owed and len(want) < min(most, free.size) and free[len(want)] < p:
                        want.append((int(p), int(free[len(want)])))
                assert list(zip(src.tolist(), dst.tolist())) == want
                held[dst] = True
                owed += src.tolist()
            elif owed:
                a.give(np.array(owed, np.int32), defer=False)
                held[owed] = False
                owed = []
            assert a.holders(range(n)).tolist() == held.astype(int).tolist()
        a.close()


def test_pending_gives_cost_alike_however_many_there_are():
    import time
    E = pkv.EventOps

    def record(ctx, stream, ev):
        ev[0] = 1
        return 0

    ops = E(E.RECORD(record), E.QUERY(lambda ctx, ev: 1), E.DESTROY(lambda ctx, ev: None), None)
    took = {}
    for n in (2000, 20000):
        a = _arena(n)
        a.set_event_ops(ops)
        ids = a.take(n)
        start = time.perf_counter()
        for i in range(n):
            a.give(ids[i:i + 1], stream=1)
        took[n] = time.perf_counter() - start
        assert a.holders(ids).sum() == 0 and a.info()[1] == 0
        a.close()
    assert took[20000] < 40 * took[2000], took     # ten times as many gives; all moved at each, it was 70 times and more
