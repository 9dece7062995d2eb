"""Rows of one request whose windows do not meet: the pages between them, before the first
window and behind the last are under no window, and a page table may hold anything there (a
cache that slides gives them back).  Every head layout that a kernel is chosen for."""
import pytest

from tests import test_gpu_attention as B

pytestmark = pytest.mark.gpu

PAGE = 64
# windows of consecutive rows of a request of 700 positions
ROWS = [[(0, 64), (256, 320)],
        [(256, 320), (0, 64)],
        [(0, 64), (64, 100), (300, 301), (640, 700)],
        [(130, 190), (0, 0), (600, 700), (600, 699)],
        [(5, 5), (400, 420), (64, 65), (420, 460), (640, 641)],
        [(i * 150, i * 150 + 3) for i in range(5)] + [(i * 150, i * 150 + 64) for i in range(4, -1, -1)],
        [(70, 100), (99, 128), (128, 192), (448, 640), (200, 256)]]


@pytest.mark.parametrize("junk", [-1, 10 ** 6, -2 ** 31, 2 ** 31 - 1])
@pytest.mark.parametrize("heads,dim", [((8, 2), 64), ((8, 2), 128), ((8, 2), 256), ((1, 1), 64), ((64, 1), 64), ((32, 2), 128),
                                       ((64, 1), 128), ((3, 3), 256)])
def test_pages_under_no_window(heads, dim, junk):
    wins = [(i, *w) for i, rows in enumerate(ROWS) for w in rows]
    c = B.Case([700] * len(ROWS), wins, *heads, dim)
    for i, rows in enumerate(ROWS):
        seen = {x // PAGE for a, b in rows for x in range(a, b)}
        for j in range(c.mp):
            if j not in seen:
                c.table[i, j] = junk
    rows = c.table.cpu().clamp(0, c.np_ - 1)
    assert B.run_paged(c) == 0
    c.table.copy_(rows)      # (for the plain form's look at the pages)
    c.check()


@pytest.mark.parametrize("heads,dim", [((8, 2), 64), ((8, 2), 128), ((8, 2), 256), ((64, 1), 128)])
def test_pages_under_a_window_still_have_to_be_there(heads, dim):
    for j in (0, 5):
        c = B.Case([700], [(0, 0, 64), (0, 300, 350)], *heads, dim)
        c.table[0, j] = -1
        assert B.run_paged(c) == B.INVALID_PAGE
        assert bool(c.out.isnan().all())
    c = B.Case([700], [(0, 0, 64), (0, 300, 350)], *heads, dim)
    c.table[0, 1:4] = -1
    c.table[0, 6:] = -1
    assert B.run_paged(c) == 0


@pytest.mark.parametrize("heads,dim", [((8, 2), 64), ((8, 2), 128), ((8, 2), 256), ((64, 1), 128)])
def test_weights_of_windows_apart(heads, dim):
    import torch
    wins = [(i, *w) for i, rows in enumerate(ROWS) for w in rows]
    c = B.Case([700] * len(ROWS), wins, *heads, dim)
    wout = torch.full((len(ROWS), c.mp * PAGE), 7.0, device="cuda")
    assert B.run_paged(c, weight_out=wout) == 0
    c.check()
    tot, bound = B._want_weights(c, None)
    assert bool(((wout.double() - tot).abs() <= bound).all())
