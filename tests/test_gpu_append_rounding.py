"""Rotating on the way to 4 bits, rounding by rounding: inputs whose code changes if a product and the sum that takes it are
rounded together.  Each of a rotation's two products and their sum is rounded by itself, so that a code does not depend on
which kernel writes it."""
import numpy as np
import pytest

from tests import append_ref as A
from tests.test_gpu_append import Case

DIM, FIXED = 64, (0, 16)              # pairs that hold a 4, so that both blocks' scales are 1
BORDERS = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0])


def code(y):
    """The value of y's code, of a block whose scale is 1."""
    d = np.abs(np.abs(y.astype(np.float64))[:, None] - A.E2M1)
    d = d + np.array([0, 1e-12] * 4)  # of two that are equally near the even one
    return np.copysign(A.E2M1[d.argmin(1)], y)


def borderline(n, dtype, seed):
    """n pairs (a, b) with angles (c, s), in turn ones where a c - b s and ones where b c + a s lies so near a border that its
    code tells three roundings from two, whichever product is not rounded."""
    import torch
    rng, f = np.random.default_rng(seed), np.float32
    got = []
    for upper in (False, True):
        m = 60000
        rounded = lambda x: torch.from_numpy(x).to({"bf16": torch.bfloat16, "f16": torch.float16}[dtype]).float().numpy()
        a, b = (rounded(rng.uniform(0.5, 2, m) * rng.choice([-1, 1], m)) for _ in range(2))
        s = rng.uniform(-1, 1, m).astype(f)
        t = rng.choice(BORDERS, m) * rng.choice([-1, 1], m)
        x, o = (b, a) if upper else (a, -b)          # y = x c + o s
        c = ((t - o.astype(np.float64) * s) / x).astype(f)
        p, q = x * c, o * s
        wide = lambda x, y, z: (x.astype(np.float64) * y + z).astype(f)
        three = code(p + q)
        other = b * c + a * s if not upper else a * c - b * s
        fits = (np.abs(c) < 4) & (np.abs(other) < 5.5) & (np.abs(p + q) < 5.5)
        for two in (code(wide(x, c, q)), code(wide(o, s, p))):
            at = np.flatnonzero(fits & (three != two))[:n // 4]
            assert len(at) == n // 4, (upper, len(at))
            got.append((a[at], b[at], c[at], s[at]))
    return [np.concatenate(z).reshape(4, -1).T.reshape(-1) for z in zip(*got)]   # the four kinds in turn


def inputs(dtype, pairs):
    """Heads [60, DIM] and their angles [60, 2, DIM / 2]."""
    n = 60
    a, b, c, s = (x.reshape(n, DIM // 2 - 2) for x in borderline(n * (DIM // 2 - 2), dtype, 5))
    free = [j for j in range(DIM // 2) if j not in FIXED]
    x, angles = np.zeros((n, DIM), np.float32), np.zeros((n, 2, DIM // 2), np.float32)
    i, j = A._pairs(DIM, 0, pairs)
    x[:, i[free]], x[:, j[free]] = a, b
    angles[:, 0, free], angles[:, 1, free] = c, s
    for k in FIXED:
        x[:, i[k]], x[:, j[k]], angles[:, 0, k] = 4, -4, 1
    return x, angles


@pytest.mark.parametrize("pairs", [False, True])
def test_the_inputs_tell_the_roundings_apart(pairs):
    x, angles = inputs("bf16", pairs)
    idx, scale = A.quantise(A.turned32(x[:, None], None, 0, angles[:, 0], angles[:, 1], 0, pairs)[:, 0])
    assert (scale == 127).all()
    i, j = A._pairs(DIM, 0, pairs)
    c, s = angles[:, 0].astype(np.float64), angles[:, 1].astype(np.float64)
    once = x.astype(np.float64)
    once[:, i], once[:, j] = x[:, i] * c - x[:, j] * s, x[:, j] * c + x[:, i] * s
    assert (A.values(A.quantise(once.astype(np.float32))[0], scale) != A.values(idx, scale)).sum() > 400


@pytest.mark.gpu
@pytest.mark.parametrize("rows", [60, 6000])      # one chunk a warp, and the kernel for many
@pytest.mark.parametrize("pairs", [False, True])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_products_and_sums_are_rounded_one_by_one(dtype, pairs, rows):
    import torch
    x, angles = inputs(dtype, pairs)
    again = np.arange(rows) % len(x)
    c = Case([(0, p) for p in range(rows)], 1, 1, DIM, dtype, True, norm=None, rot=DIM, pairs=pairs, q4=True, values=False, nr=1,
             mp=-(-rows // 64))
    assert c.rope.shape[0] >= rows
    c.rope[:rows] = torch.from_numpy(angles[again]).cuda()
    for t in (c.q, c.k):
        t[:, 0] = torch.from_numpy(x[again]).to(t.dtype).cuda()
    assert c.run() == 0
    c.check()
