"""The host's count of a cache's pages (uw_pages) against a dictionary (CPU)."""
import ctypes as C

import numpy as np
import pytest

import decode_gemm_bf16_amd as uw


def refused(status, f, *args):
    with pytest.raises(uw.UwError) as e:
        f(*args)
    assert e.value.status == status


def test_by_hand():
    p = uw.Pages(6)
    a = p.take(4)
    assert a.tolist() == [0, 1, 2, 3] and p.left == 2 and p.holders(3) == 1 and p.holders(4) == 0
    p.share(a[:3])  # a fork shares three pages
    assert p.own(2) == 4 and p.holders(2) == 1 and p.holders(4) == 1  # its partial page becomes its own
    assert p.own(2) == 2
    refused(uw.ERR_OOM, p.take, 2)
    assert p.left == 1
    p.drop(a)
    assert [p.holders(i) for i in range(6)] == [1, 1, 0, 0, 1, 0]
    src, dst = p.compact()
    assert src.tolist() == [4] and dst.tolist() == [2] and p.left == 3
    assert p.take(3).tolist() == [3, 4, 5] and p.left == 0
    refused(uw.ERR_OOM, p.take, 1)
    p.share([0])
    refused(uw.ERR_OOM, p.own, 0)
    assert p.holders(0) == 2 and p.take(0).size == 0


def test_refusals_change_nothing():
    p = uw.Pages(4)
    p.take(2)
    p.share([1])
    for f, list_ in ((p.share, [0, 2]), (p.share, [-1]), (p.share, [4]), (p.drop, [0, 0]), (p.drop, [1, 1, 1]), (p.drop, [3]),
                     (p.drop, [1, 2 ** 31 - 1])):
        refused(uw.ERR_INVALID_ARG, f, list_)
    refused(uw.ERR_INVALID_ARG, p.own, 2)
    refused(uw.ERR_INVALID_ARG, p.take, -1)
    assert [p.holders(i) for i in range(4)] == [1, 2, 0, 0]
    p.drop([1, 0, 1])
    assert p.left == 4
    refused(uw.ERR_INVALID_ARG, uw.Pages, 0)
    refused(uw.ERR_INVALID_ARG, uw.Pages, (1 << 26) + 1)
    L, i, n = uw._lib, C.c_int32(), C.c_int64()
    h = C.c_void_p()
    assert L.uw_pages_create(4, None) == uw.ERR_INVALID_ARG
    assert L.uw_pages_take(None, 1, C.addressof(i)) == uw.ERR_INVALID_ARG
    assert L.uw_pages_take(p._h, 1, None) == L.uw_pages_own(p._h, 0, None) == uw.ERR_INVALID_ARG
    assert L.uw_pages_compact(p._h, None, None, C.byref(n)) == uw.ERR_INVALID_ARG
    assert L.uw_pages_left(None) == L.uw_pages_holders(None, 0) == 0
    L.uw_pages_free(None)
    assert not h.value


@pytest.mark.parametrize("seed", range(4))
def test_against_a_dictionary(seed):
    rng = np.random.default_rng(seed)
    size = int(rng.integers(20, 200))
    p, held, tables = uw.Pages(size), {}, []
    for _ in range(400):
        what = rng.random()
        free = [i for i in range(size) if i not in held]
        if what < 0.35:
            n = int(rng.integers(0, 8))
            if n > len(free):
                refused(uw.ERR_OOM, p.take, n)
            else:
                t = p.take(n).tolist()
                assert t == free[:n]
                held.update({i: 1 for i in t})
                tables.append(t)
        elif what < 0.55 and tables:
            t = list(tables[rng.integers(len(tables))])
            p.share(t)
            for i in t:
                held[i] += 1
            tables.append(t)
        elif what < 0.8 and tables:
            t = tables.pop(rng.integers(len(tables)))
            p.drop(t)
            for i in t:
                held[i] -= 1
                if held[i] == 0:
                    del held[i]
        elif what < 0.95 and tables:
            t = tables[rng.integers(len(tables))]
            if t:
                if held[t[-1]] == 1:
                    assert p.own(t[-1]) == t[-1]
                elif not free:
                    refused(uw.ERR_OOM, p.own, t[-1])
                else:
                    held[t[-1]] -= 1
                    t[-1] = p.own(t[-1])
                    assert t[-1] == free[0]
                    held[t[-1]] = 1
        else:
            src, dst = p.compact()
            used = len(held)
            assert src.tolist() == sorted(i for i in held if i >= used)
            assert dst.tolist() == [i for i in range(used) if i not in held]
            name = dict(zip(src.tolist(), dst.tolist()))
            held = {name.get(i, i): c for i, c in held.items()}
            tables = [[name.get(i, i) for i in t] for t in tables]
        assert p.left == size - len(held)
        assert all(p.holders(i) == held.get(i, 0) for i in range(size))
