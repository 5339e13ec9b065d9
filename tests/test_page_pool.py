"""The page pool's counting on the host (CPU only; copies are recorded, not made)."""
import random

import pytest
import torch

from sparse_weight_direct_amd import cache


@pytest.fixture
def copies(monkeypatch):
    made = []

    def copy(pool, source, target, *, stream=None):
        s, t = source.tolist(), target.tolist()
        assert len(set(t)) == len(t) and not set(s) & set(t)
        made.append((s, t))
        pool[:, t] = pool[:, s]  # as the launch does
        return pool

    monkeypatch.setattr(cache, "cache_copy", copy)
    return made


def _pool(pages=10, **kw):
    return cache.PagePool(2, pages, 1, 8, page_size=16, device="cpu", **kw)


def test_extend_fork_free(copies):
    p = _pool()
    a = p.add()
    table, past = p.extend([a], [20])
    assert table.tolist() == [[0, 1]] and past.tolist() == [0] and p.length(a) == 20 and p.free_pages == 8
    b = p.fork(a)
    assert p.table([a, b]).tolist() == [[0, 1], [0, 1]] and p.free_pages == 8 and not copies
    table, past = p.extend([b], [1])  # its last page is a's too
    assert table.tolist() == [[0, 2]] and past.tolist() == [20] and copies == [([1], [2])]
    table, past = p.extend([a, b], [13, 0], width=4)  # now it is its own
    assert table.tolist() == [[0, 1, 3, -1], [0, 2, -1, -1]] and past.tolist() == [20, 21] and len(copies) == 1
    p.free(a)
    assert p.free_pages == 8 and p.table([b]).tolist() == [[0, 2]]
    p.free(b)
    assert p.free_pages == 10


def test_two_forks_extended_together_need_one_copy(copies):
    p = _pool()
    a = p.add()
    p.extend([a], [5])
    b = p.fork(a)
    table, _ = p.extend([a, b], [1, 1])
    assert len(copies) == 1 and len(copies[0][0]) == 1
    assert len({row[0] for row in table.tolist()}) == 2 and p.free_pages == 8


def test_a_full_last_page_is_shared_without_a_copy(copies):
    p = _pool()
    a = p.add()
    p.extend([a], [16])
    b = p.fork(a)
    assert p.extend([a, b], [1, 1])[0].tolist() == [[0, 1], [0, 2]] and not copies
    c = p.fork(a)
    p.extend([c], [0])
    assert not copies


def test_too_few_pages_changes_nothing(copies):
    p = _pool(pages=3)
    a = p.add()
    p.extend([a], [20])
    b = p.fork(a)
    before = (list(p._free), list(p._users), p.table([a, b]).tolist())
    with pytest.raises(MemoryError):
        p.extend([b, a], [13, 20])
    with pytest.raises(ValueError):
        p.extend([a], [40], width=2) if p.free_pages >= 2 else p.extend([a], [1], width=1)
    with pytest.raises(ValueError):
        p.extend([a, a], [1, 1])
    with pytest.raises(ValueError):
        p.extend([a], [-1])
    with pytest.raises(ValueError):
        p.table([a], width=1)
    with pytest.raises(KeyError):
        p.extend([99], [1])
    assert before == (list(p._free), list(p._users), p.table([a, b]).tolist()) and not copies
    for bad in (dict(pages=0), dict(page_size=48)):
        with pytest.raises(ValueError):
            cache.PagePool(1, bad.get("pages", 4), 1, 8, page_size=bad.get("page_size", 16), device="cpu")


def test_forget_and_compact(copies):
    p = _pool()
    a, b = p.add(), p.add()
    p.extend([a, b], [40, 40])  # pages 0 1 2 and 3 4 5
    p.forget(a, 33)
    assert p.table([a]).tolist() == [[-1, -1, 2]] and p.free_pages == 6
    c = p.fork(a)
    p.forget(a, 33)  # once is enough
    assert p.compact() == 4 and p.free_pages == 6
    assert p.table([a, b, c]).tolist() == [[-1, -1, 2], [3, 0, 1], [-1, -1, 2]]
    assert p.compact() == 4
    p.free(a)
    p.free(c)
    p.free(b)
    assert p.compact() == 0 and p.free_pages == 10 and sorted(p._free) == list(range(10))


def test_random_walk_keeps_every_sequence(copies):
    """Sequences write their own numbers into their pages; whatever happens, each finds its own."""
    rng = random.Random(4)
    p = _pool(pages=40, dtype=torch.float64)
    want: dict[int, list[float]] = {}
    for step in range(600):
        op = rng.choice(["add", "extend", "extend", "extend", "fork", "free", "compact"])
        if op == "add" and len(want) < 12:
            want[p.add()] = []
        elif op == "fork" and want and len(want) < 12:
            s = rng.choice(list(want))
            want[p.fork(s)] = list(want[s])
        elif op == "free" and want:
            s = rng.choice(list(want))
            p.free(s)
            del want[s]
        elif op == "compact":
            used = p.compact()
            assert used == p.pages - p.free_pages
            assert all(x < used for s in want for x in p.table([s])[0].tolist())
        elif op == "extend" and want:
            some = rng.sample(list(want), rng.randint(1, min(3, len(want))))
            n = [rng.randint(0, 30) for _ in some]
            try:
                table, past = p.extend(some, n)
            except MemoryError:
                continue
            for row, t0, s, k in zip(table.tolist(), past.tolist(), some, n):
                assert t0 == len(want[s])
                for t in range(t0, t0 + k):
                    v = float(rng.random())
                    p.k_pages(1)[row[t // 16], 0, t % 16] = v
                    want[s].append(v)
        users = [0] * 40
        for s, values in want.items():
            assert p.length(s) == len(values)
            row = p.table([s])[0].tolist()
            for page in row:
                if page >= 0:
                    users[page] += 1
            got = [float(p.k_pages(1)[row[t // 16], 0, t % 16, 3]) for t in range(len(values))]
            assert got == values
        assert users == p._users and p.free_pages == users.count(0)
    assert any(copies)
