"""Slots named twice among more rows than the table of slots holds: a bitmap finds them, sized by the pool, a part of it at a
time where the pool is large.  Slots that the bitmap keeps in one word, in its last part, and calls that are mostly padding."""
import numpy as np
import pytest

from tests.test_gpu_append import INVALID_PAGE, PAGE, Case

pytestmark = pytest.mark.gpu

MOST = 1 << 14                        # rows that the table holds


def call(pages, slots, rows, seed):
    """`rows` rows, the first ones with these slots, the others not there; one request that has all pages, in any order."""
    table = np.random.default_rng(seed).permutation(pages).astype(np.int32)
    at = np.argsort(table)[slots // PAGE] * PAGE + slots % PAGE
    where = np.random.default_rng(seed + 1).permutation(rows)[:len(slots)]     # the rows that are there
    pos = np.full(rows, -1)
    pos[where] = at
    c = Case([(0, int(p)) for p in pos], 0, 1, 64, "f16", True, norm=None, table=table[None], pages=pages, nr=1, mp=pages, values=False)
    return c, where, at


def same(c):
    return all(bool((a == b).all()) for a, b in zip(c.caches, c.before))


def check(pages, slots, rows, twice, seed=3):
    """Nothing is named twice; then the rows of each pair (i, j) of `twice` name one slot."""
    c, where, at = call(pages, slots, rows, seed)
    assert c.run() == 0
    c.check()
    c.before = [x.clone() for x in c.caches]
    c.k.zero_()
    for i, j in twice:
        c.pos[int(where[j])] = int(at[i])
        assert c.run() == INVALID_PAGE, (i, j)
        assert same(c), (i, j)
        c.pos[int(where[j])] = int(at[j])
    assert c.run() == 0               # (and each of them alone is fine again)


@pytest.mark.parametrize("pages", [257, 300, 1100, 5000, 16385, 40000])
@pytest.mark.parametrize("step", [1, 1 << 10, 1 << 12, 1 << 15])
def test_slots_of_one_word(pages, step):
    """Neighbours, and slots that are `step` apart: the bitmap's bits of a word are 2^10 to 2^15 slots apart."""
    n, total = MOST + 40, pages * PAGE
    order = np.arange(total)
    order = order[np.lexsort((order // step, order % step))]     # 0, step, 2 step, ..., 1, 1 + step, ...
    check(pages, order[:n], n, [(0, 1), (n - 1, 0), (5, n // 2)])


@pytest.mark.parametrize("pages", [16385, 16400, 40000])
def test_the_last_part(pages):
    """A bitmap holds 2^20 slots: the first and last of each part, and of the last, which is not full."""
    total, part = pages * PAGE, 1 << 20
    ends = sorted({x for p in range(0, total, part) for x in (p, p + 1, min(p + part, total) - 1)})
    rng = np.random.default_rng(pages)
    some = np.setdiff1d(rng.permutation(total)[:MOST + 100], ends)[:MOST + 1]
    slots = np.concatenate([ends, some]).astype(np.int64)
    last = len(ends) - 1
    check(pages, slots, len(slots), [(0, last), (last, 0), (last, len(slots) - 1), (1, 2), (last - 1, last)])


@pytest.mark.parametrize("pages", [1, 3, 32, 33, 40, 250])
def test_mostly_padding(pages):
    """Rows that are not there choose the bitmap too; a pool of few slots has a small one."""
    total = pages * PAGE
    slots = np.random.default_rng(pages).permutation(total)[:max(2, total - 5)]
    check(pages, slots, MOST + 1, [(0, 1), (len(slots) - 1, 0)])
    check(pages, slots, MOST + 500, [(len(slots) // 2, 0)])
