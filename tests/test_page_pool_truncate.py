"""Taking back what extend() promised: a sequence whose call was refused is as it was before (CPU only)."""
import random

import pytest

from test_page_pool import _pool, copies  # noqa: F401


def test_a_refused_extension_is_taken_back(copies):  # noqa: F811
    p = _pool()
    a, b = p.add(), p.add()
    p.extend([a, b], [20, 3])
    before = p.table([a, b]).tolist(), p.free_pages
    for n in ([1, 1], [12, 13], [13, 14], [30, 0], [0, 60]):
        p.extend([a, b], n)
        p.truncate(a, 20)
        p.truncate(b, 3)
        assert (p.table([a, b]).tolist(), p.free_pages) == before and p.length(a) == 20 and p.length(b) == 3
        assert p.extend([a, b], [0, 0])[1].tolist() == [20, 3]
    p.truncate(a, 16)
    assert p.table([a]).tolist() == [[0]] and p.length(a) == 16 and p.free_pages == before[1] + 1
    p.truncate(a, 16)
    p.truncate(a, 0)
    assert p.table([a]).tolist() == [[-1]] and p.length(a) == 0
    assert p.extend([a], [1])[1].tolist() == [0]


def test_shared_pages_stay_the_others(copies):  # noqa: F811
    p = _pool()
    a = p.add()
    p.extend([a], [40])
    b = p.fork(a)
    p.extend([b], [1])  # its last page is its own now
    assert copies == [([2], [3])]
    p.truncate(b, 40)
    p.truncate(b, 20)  # inside a page that a has too
    assert p.table([a, b]).tolist() == [[0, 1, 2], [0, 1, -1]] and p.free_pages == 7
    assert p.extend([b], [1])[0].tolist() == [[0, 3]] and len(copies) == 2  # so it is copied before it is written
    p.free(a)
    p.free(b)
    assert p.free_pages == 10


def test_truncations_that_are_refused(copies):  # noqa: F811
    p = _pool()
    a = p.add()
    p.extend([a], [50])
    p.forget(a, 33)
    before = p.table([a]).tolist(), p.free_pages
    for n in (-1, 51, 20, 31):  # 20 and 31 lie in pages that are gone
        with pytest.raises(ValueError):
            p.truncate(a, n)
    with pytest.raises(KeyError):
        p.truncate(7, 0)
    assert (p.table([a]).tolist(), p.free_pages) == before and p.length(a) == 50
    p.truncate(a, 32)  # the next position opens a page of its own
    assert p.table([a]).tolist() == [[-1, -1]] and p.extend([a], [1])[0][0, 2] >= 0


def test_random_extensions_and_truncations_keep_the_count(copies):  # noqa: F811
    rng = random.Random(9)
    p = _pool(pages=60)
    ids = []
    for _ in range(800):
        op = rng.choice(["add", "extend", "extend", "truncate", "truncate", "fork", "free", "compact"])
        if op == "add" and len(ids) < 10:
            ids.append(p.add())
        elif op == "fork" and ids and len(ids) < 10:
            ids.append(p.fork(rng.choice(ids)))
        elif op == "free" and ids:
            p.free(ids.pop(rng.randrange(len(ids))))
        elif op == "compact":
            p.compact()
        elif op == "extend" and ids:
            s, n = rng.choice(ids), rng.randint(0, 40)
            try:
                assert p.extend([s], [n])[1].tolist() == [p.length(s) - n]
            except MemoryError:
                pass
        elif op == "truncate" and ids:
            s = rng.choice(ids)
            p.truncate(s, rng.randint(0, p.length(s)))
        users = [0] * 60
        for s in ids:
            row = [x for x in p.table([s])[0].tolist() if x >= 0]
            assert len(row) == -(-p.length(s) // 16)
            for page in row:
                users[page] += 1
        assert users == p._users and p.free_pages == users.count(0) and sorted(p._free) == [i for i in range(60) if not users[i]]
