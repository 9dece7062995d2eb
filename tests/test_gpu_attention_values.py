"""Attention where the scores or the softmax weights reach the ends of their types: one position
far above a long tail (fp16 weights lose bits below 2^-14 and vanish below 2^-25), scores beyond
2^24, scores of +infinity.  Every kernel, whole and cut units, windows and lists of slots."""
import math

import pytest

from tests import attn_ref as A
from tests import test_gpu_attention as B

pytestmark = pytest.mark.gpu

PAGE = 64
# (query heads, key-value heads), head dimension, rows of the request
KINDS = [((8, 2), 64, 1), ((8, 2), 128, 3), ((8, 2), 256, 1), ((64, 1), 128, 1), ((64, 1), 128, 2), ((32, 8), 128, 1),
         ((40, 1), 64, 2)]


def _attend(c, form):
    """Runs the case over its windows, or over the same positions as lists of slots."""
    import torch
    import fp4_sparse_attention_tma_gb300 as m
    if form == "paged":
        assert B.run_paged(c) == 0
        return
    n = int(c.end.max())
    pos = torch.arange(n, device="cuda")
    slots = (c.table.long()[c.req.long()][:, pos // PAGE] * PAGE + pos % PAGE)
    slots = torch.where(pos < c.end[:, None], slots, -1).to(torch.int32)
    assert m.idx_attn_selected(c.q, c.k, c.v, slots, c.scale, c.out, out_lse=c.lse) == 0
    torch.cuda.synchronize()


def _place(c, i, pos):
    import torch
    pos = torch.as_tensor(pos)
    return c.table.cpu()[i][pos // PAGE].long().cuda(), (pos % PAGE).cuda()


def _case(n, kind, dtype, copies=1):
    """`copies` requests that share the pages of one: with many of them a worker sees whole requests (one
    alone is divided among all workers, each with a maximum of its own)."""
    import torch
    heads, dim, rows = kind
    c = B.Case([n], [(0, 0, n)] * (rows * copies), *heads, dim, dtype)
    c.table = c.table.expand(copies, -1).contiguous()
    c.req = torch.arange(copies, dtype=torch.int32, device="cuda").repeat_interleave(rows)
    c.wins = [(int(i), 0, n) for i in c.req.cpu()]
    return c


def _many(kind):
    """Requests that give every worker of the kernel more than one unit."""
    return {(64, 1): 200, (32, 8): 38}.get(kind[0], 1300)


# ------------------------------------------------------------- weights ----

@pytest.mark.parametrize("form", ["paged", "slots"])
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_long_tail_under_one_position(kind, dtype, form):
    """Position j weighs 1 and every other 2^-d: out = (v_j + (n - 1) 2^-d v) / (1 + (n - 1) 2^-d).

    The scores are exact products.  A weight is rounded to the inputs' type with a relative error
    of u; an fp16 weight is taken relative to at least 2^10 times the row's largest, so that one
    below fp16's normal range is off by 2^-25 2^-10 of it at the most, and the output by n times
    that: no more than 2^-17 of max |v| for the longest row here."""
    import torch
    u = 2.0 ** -8 if dtype == "bf16" else 2.0 ** -11
    many = _many(kind)
    for n, d, copies in ((5001, 10.3, many), (5001, 17.45, many), (5001, 20.55, many), (5001, 24.7, many), (5001, 25.3, many),
                         (5001, 26.4, many), (1900, 24.85, many), (262143, 24.6, 1), (262143, 25.4, 1)):
        if n > 100000 and (kind[0][1] > 2 or kind[1] > 128):
            continue
        c = _case(n, kind, dtype, copies)
        D = c.dim
        # q = e_0: the score is scale * log2(e) * k_0 in units of log2
        c.q.zero_()
        c.q[:, :, 0] = 1.0
        c.k.zero_()
        j = {0: 0, 1: n - 1, 2: n // 2}[int(d * 10) % 3]
        c.k[(*_place(c, 0, [j]), slice(None), 0)] = 64.0
        c.scale = d * math.log(2) / 64.0
        # signs that agree, then values that cancel; the heavy position's value is 0
        for signs in (False, True):
            pos = torch.arange(n)
            page, off = _place(c, 0, pos)
            v = torch.ones(n, device="cuda")
            if signs:
                v[1::2] = -0.5
            c.v[page, off] = v.to(c.v.dtype)[:, None, None].expand(n, c.hk, D)
            c.v[_place(c, 0, [j])] = 0.0
            v[j] = 0.0
            _attend(c, form)
            w = torch.full((n,), 2.0 ** -d, dtype=torch.float64, device="cuda")
            w[j] = 1.0
            total = w.sum()
            want, mag = float((w * v.double()).sum() / total), float((w * v.abs().double()).sum() / total)
            # fp32: the scale, its product with log2(e) and the score's are rounded, as are 2^x and the sums
            ep = 2 * (d * 3 * 2.0 ** -24 * math.log(2)) + 2.0 ** -20
            bound = u * abs(want) + (u + ep + n * 2.0 ** -24) * mag + (n * 2.0 ** -35 if dtype == "f16" else 0.0)
            if dtype == "f16" and abs(want) < 2.0 ** -14:
                bound += 2.0 ** -25      # the output's own rounding
            err = float((c.out.double() - want).abs().max())
            assert err <= bound, (n, d, signs, want, err, bound)
            # (n additions to the sum)
            assert float((c.lse.double() - (d * math.log(2) + math.log(total))).abs().max()) <= 2.0 ** -17 + n * 2.0 ** -24


@pytest.mark.parametrize("kind", KINDS)
def test_random_tail_under_one_position_f16(kind):
    """Scores of deviation 1/2 and one position 16 to 18 above them, first, last or between."""
    import torch
    for n, gap in ((30000, 16.0), (30000, 17.0), (30000, 18.0)):
        c = _case(n, kind, "f16", _many(kind) // 4)
        j = {16.0: 0, 17.0: 31, 18.0: 1234}[gap]
        # every head's queries are parallel to the unit vector x, whose keys carry the scores
        x = torch.ones(c.dim, device="cuda") / 8.0
        c.q[:] = x.half()
        g = torch.Generator(device="cuda")
        g.manual_seed(int(gap))
        s = torch.randn(n, c.hk, device="cuda", generator=g) * 0.5
        s[j] = gap
        c.scale = 1.0
        page, off = _place(c, 0, torch.arange(n))
        c.k[page, off] = (s[:, :, None] * (8.0 / c.dim)).half().expand(n, c.hk, c.dim)
        c.v[_place(c, 0, [j])] = 0.001
        c.v.abs_()                       # values of one sign: errors of the weights add up
        assert B.run_paged(c) == 0
        k, v = c.rows()[0]
        want, lse, _, _, bl, ep = A.attend(c.q[0], k, v, c.scale)     # (every row's)
        u = 2.0 ** -11
        bound = u * want + (u + ep[:, None] + n * 2.0 ** -24) * want + n * 2.0 ** -35 * float(v.max())   # all values are positive
        err = (c.out.double() - want).abs()
        assert bool((err <= bound).all()), (gap, float((err / want).max()), float((bound / want).max()))
        assert bool(((c.lse.double() - lse).abs() <= bl + n * 2.0 ** -24).all())


# -------------------------------------------------------- large scores ----

@pytest.mark.parametrize("form", ["paged", "slots"])
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_scores_beyond_2_to_24(kind, dtype, form):
    """Scores whose fp32 neighbours are far apart: the largest still weighs 1, and two that are
    equal weigh half each.  Queries and keys have few bits, so the products are exact; the
    others' scores lie lower by more than 2^7."""
    import torch
    for n in (3, 130, 5000):
        for e in (5, 8, 12, 15):               # q . k = D 2^2e 1.2109375 1.4140625
            for extra in (1.0, 1.3, 1.7):
                c = _case(n, kind, dtype)
                c.scale = extra * c.dim ** -0.5
                c.q.fill_(2.0 ** e * 1.2109375)
                c.k.fill_(0.0)
                c.k[_place(c, 0, [1])] = 2.0 ** e * 1.4140625
                c.k[_place(c, 0, [n - 1])] = 2.0 ** e * 1.4140625
                _attend(c, form)
                s = 2.0 ** (2 * e) * 1.2109375 * 1.4140625 * c.dim * float(torch.tensor(c.scale, dtype=torch.float32))
                _, v = c.rows()[0]
                want = (0.5 * (v[1].double() + v[n - 1].double()))
                got = c.out.double().view(-1, c.hk, c.hq // c.hk, c.dim)
                u = 2.0 ** -8 if dtype == "bf16" else 2.0 ** -11
                # (weights of 1/2 after the division: exact; the output's rounding, and 2^-20 of fp32)
                assert bool(((got - want[None, :, None]).abs() <= (u + 2.0 ** -20) * want.abs()[None, :, None] + 2.0 ** -20).all()), (n, e, extra)
                assert bool(((c.lse.double() - (s + math.log(2))).abs() <= 2.0 ** -21 * s).all()), (n, e, extra)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_weights_of_scores_beyond_2_to_24(kind, dtype):
    import torch
    for n in (130, 5000):
        for e in (8, 12, 15):
            c = _case(n, kind, dtype)
            c.q.fill_(2.0 ** e * 1.2109375)
            c.k.fill_(0.0)
            c.k[_place(c, 0, [77])] = 2.0 ** e * 1.4140625
            w = torch.full((1, c.mp * PAGE), 7.0, device="cuda")
            assert B.run_paged(c, weight_out=w) == 0
            want = torch.zeros_like(w)
            want[0, 77] = c.hq * len(c.wins)
            assert bool(((w - want).abs() <= 2.0 ** -18 * want).all()), (n, e)


# ------------------------------------------------------------ infinity ----

@pytest.mark.parametrize("form", ["paged", "slots"])
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_scores_of_plus_infinity(kind, dtype, form):
    """A visible score of +infinity: log sum exp is +infinity and the outputs are NaN, as in the
    formula; with a visible score of NaN as well, both are NaN.  Other requests notice nothing."""
    import torch
    heads, dim, rows = kind
    for n in (1, 40, 300, 9000):
        for j in sorted({0, n // 2, n - 1}):
            c = B.Case([n, 500], [(0, 0, n)] * rows + [(1, 0, 500)] * rows, *heads, dim, dtype)
            c.q.abs_().clamp_(min=0.125)
            _attend(c, form)
            out, lse = c.out.clone(), c.lse.clone()
            c.k[(*_place(c, 0, [j]), slice(None), 3)] = float("inf")
            _attend(c, form)
            assert bool(torch.isposinf(c.lse[:rows]).all()), (n, j)
            assert bool(c.out[:rows].isnan().all()), (n, j)
            assert bool((c.out[rows:] == out[rows:]).all()) and bool((c.lse[rows:] == lse[rows:]).all())
            # one more far from it, and then a score of NaN
            c.k[(*_place(c, 0, [n - 1 - j]), slice(None), 3)] = float("inf")
            _attend(c, form)
            assert bool(torch.isposinf(c.lse[:rows]).all()) and bool(c.out[:rows].isnan().all()), (n, j)
            if n > 2:
                for x in {1, n - 2}:
                    k0 = c.k.clone()
                    c.k[(*_place(c, 0, [x]), slice(None), 5)] = float("nan")
                    _attend(c, form)
                    assert bool(c.lse[:rows].isnan().all()) and bool(c.out[:rows].isnan().all()), (n, j, x)
                    c.k.copy_(k0)


@pytest.mark.parametrize("form", ["paged", "slots"])
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_plus_infinity_within_a_workers_range(kind, dtype, form):
    """The same where one worker sees all of a request: before, among and after finite scores."""
    import torch
    for n, at in ((700, [0]), (700, [350]), (700, [699]), (2100, [5, 2000])):
        c = _case(n, kind, dtype, _many(kind))
        c.q.abs_().clamp_(min=0.125)
        c.k[(*_place(c, 0, at), slice(None), 3)] = float("inf")
        _attend(c, form)
        assert bool(torch.isposinf(c.lse).all()) and bool(c.out.isnan().all()), (n, at)
        c.k[(*_place(c, 0, [300]), slice(None), 5)] = float("nan")
        _attend(c, form)
        assert bool(c.lse.isnan().all()) and bool(c.out.isnan().all()), (n, at)


@pytest.mark.parametrize("kind", KINDS)
def test_weights_beside_a_score_of_plus_infinity(kind):
    """exp(s - infinity) is 0 for the finite scores and NaN where the score is infinite."""
    import torch
    for n in (300, 9000):
        c = _case(n, kind, "bf16")
        c.q.abs_().clamp_(min=0.125)
        c.k[(*_place(c, 0, [100]), slice(None), 3)] = float("inf")
        w = torch.full((1, c.mp * PAGE), 7.0, device="cuda")
        assert B.run_paged(c, weight_out=w) == 0
        assert bool(w[0, 100].isnan())
        w[0, 100] = 0.0
        assert bool((w == 0).all())


def test_a_scale_beyond_the_kernels_units_is_refused():
    """Exponents are counted in units of log2: scale * log2(e) has to be finite."""
    import torch
    import fp4_sparse_attention_tma_gb300 as m
    c = B.Case([100], [(0, 0, 100)], 8, 2, 64)
    c.q.zero_()                  # scores of 0 at any scale: out is the mean of the values
    for scale, code in ((3.4e38, B.INVALID_ARGUMENT), (2.4e38, B.INVALID_ARGUMENT), (2.3e38, 0), (1e-45, 0)):
        c.scale = scale
        c.out.fill_(7.0)
        assert B.run_paged(c) == code
        if code:
            assert bool((c.out == 7).all())
            slots = torch.zeros(1, 4, dtype=torch.int32, device="cuda")
            assert m.idx_attn_selected(c.q, c.k, c.v, slots, scale, c.out, raise_on_error=False) == code
        else:
            c.check()
