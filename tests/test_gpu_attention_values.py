"""Attention where the scores reach the ends of their type: scores beyond 2^24.  Every kernel,
whole and cut units, windows and lists of slots."""
import math

import pytest

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
