"""Writing a paged cache where every warp has more chunks of heads than its ring holds, so that a stage is refilled while
the next chunk waits: rotations with and without a norm, whole and partial, of halves and of neighbours, in 16 bits and
in 4, with chunks that are partly filled and rows that are not there, against the plain forms and bounds of
tests/append_ref.py."""
import numpy as np
import pytest

from tests.test_gpu_append import PAGE, ROT, Case

pytestmark = pytest.mark.gpu

# A chunk is four times 32 lanes of 8 elements: 16 heads of 64, 8 of 128, 4 of 256.  Queries fill one and begin another,
# so a row has four chunks and a call 14,800, four and more for each of at most 24 warps on 152 SMs, whose rings hold two.
HEADS = {64: 17, 128: 9, 256: 5}
N, MP = 3700, 32


def some_rows(seed):
    """Rows in any order over three requests, some of them not there."""
    at = np.random.default_rng(seed).permutation(3 * MP * PAGE)[:N]
    return [(int(s) // (MP * PAGE), -1 if i % 37 == 5 else int(s) % (MP * PAGE)) for i, s in enumerate(at)]


def run(dim, rot, norm, dtype, fp4, layout="slot", in_place=False, **kw):
    n, first, pairs = rot
    n, first = (dim if n == "all" else n), (first if first >= 0 else dim + first)
    heads = kw.pop("heads", (HEADS[dim], 1))
    c = Case(some_rows(dim + n), *heads, dim, dtype, fp4, layout, norm, n, first, pairs, seed=n + first + 1, mp=MP, **kw)
    if not in_place:
        assert c.run() == 0
    else:
        keep, c.out_q = c.q.clone(), c.q
        assert c.run() == 0
        got, c.q = c.out_q.clone(), keep
        skipped = [i for i, r in enumerate(c.rows) if r[1] < 0]
        assert bool((got[skipped] == keep[skipped]).all())
        got[skipped] = 7.0
        c.out_q = got
    c.check()


@pytest.mark.parametrize("fp4", [False, True])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("rot", [("all", 0, False), (32, 8, False), (48, 16, False)])
def test_halves_without_a_norm(fp4, dtype, dim, rot):
    """Nothing but the copies' own order keeps a lane from the pieces that others still read."""
    run(dim, rot, None, dtype, fp4)


@pytest.mark.parametrize("fp4", [False, True])
@pytest.mark.parametrize("norm", [None, "same", "f32"])
@pytest.mark.parametrize("rot", range(len(ROT)))
def test_forms(fp4, norm, rot):
    i = rot + [None, "same", "f32"].index(norm)      # every rotation and norm, with every dimension, type and layout among them
    run([64, 128, 256][i % 3], ROT[rot], norm, ["bf16", "f16"][i // 3 % 2], fp4, ["slot", "head", "joint"][rot % 3])


@pytest.mark.parametrize("fp4", [False, True])
@pytest.mark.parametrize("norm", [None, "f32"])
@pytest.mark.parametrize("rot", [("all", 0, False), (32, 8, False), (64, -64, True)])
def test_queries_in_place(fp4, norm, rot):
    run(128, rot, norm, "bf16", fp4, in_place=True)


@pytest.mark.parametrize("norm", [None, "same", "f32"])
@pytest.mark.parametrize("rot", [("all", 0, False), (48, 16, False), (64, -64, True)])
def test_queries_in_4_bits(norm, rot):
    """With values and without, as the indexer's cache has none; queries of one chunk and a half."""
    run(128, rot, norm, "f16", True, q4=True, heads=(9, 1))
    run(64, rot if rot[0] != 48 else (32, 8, False), norm, "bf16", True, q4=True, heads=(5, 1), values=False)


@pytest.mark.parametrize("fp4", [False, True])
@pytest.mark.parametrize("norm", [None, "same"])
def test_without_queries(fp4, norm):
    """Two full chunks of keys and one of a single head, then those of values."""
    run(128, ("all", 0, False), norm, "bf16", fp4, heads=(0, 17))
