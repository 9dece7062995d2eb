"""What appending to 4 bits writes and attention over it refuses: an element that is not finite, or too large, of one request
among others; and the sizes of queries and keys up to which scores keep their value."""
import math

import pytest

from tests import attn4_ref as A

pytestmark = pytest.mark.gpu

PAGE, MAX_SCALE_BYTE, INVALID_VALUE = 64, 167, 10


class Chain:
    """Three requests of 100 tokens: keys and values appended to a 4-bit cache, then a row of queries a request over it."""

    def __init__(self, hq, hk, dim, seed):
        import torch
        import fp4_sparse_attention_tma_gb300 as m
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        self.m, self.n = m, 100
        u8 = lambda w: torch.zeros(6, PAGE, hk, w, dtype=torch.uint8, device="cuda")
        self.cache = [u8(dim // 2), u8(dim // 32), u8(dim // 2), u8(dim // 32)]
        i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
        self.table = i32([[4, 1], [0, 3], [5, 2]])
        self.req, self.pos = i32([r for r in range(3) for _ in range(100)]), i32(list(range(100)) * 3)
        make = lambda *s: torch.randn(*s, device="cuda", generator=g).to(torch.bfloat16)
        self.k, self.v, self.q = make(300, hk, dim), make(300, hk, dim), make(3, hq, dim)
        self.out, self.lse = torch.empty_like(self.q), torch.empty(3, hq, device="cuda")
        self.rows, self.start, self.end = i32([0, 1, 2]), i32([0] * 3), i32([100] * 3)
        self.scale = dim ** -0.5

    def append(self):
        assert self.m.idx_cache_append_fp4(self.k, self.v, self.table, self.req, self.pos, *self.cache) == 0

    def attend(self):
        return self.m.idx_attn_paged_fp4(self.q, *self.cache, self.table, self.rows, self.start, self.end, self.scale, self.out,
                                         out_lse=self.lse, raise_on_error=False)

    def at(self, r):
        import torch
        pos = torch.arange(self.n, device="cuda")
        return self.table[r].long()[pos // PAGE], pos % PAGE

    def refused(self):
        """Which requests hold a scale byte that attention refuses."""
        return [r for r in range(3) if any(bool((s[self.at(r)] > MAX_SCALE_BYTE).any()) for s in self.cache[1::2])]


@pytest.mark.parametrize("heads", [(8, 2), (64, 1)])
@pytest.mark.parametrize("value", [math.nan, math.inf, 6 * 2.0 ** 41, -7 * 2.0 ** 40])
@pytest.mark.parametrize("of_keys", [True, False])
def test_a_request_that_is_refused_is_found_by_its_scales(heads, value, of_keys):
    """Appended as it is; attention refuses the call; without the request's row the others are answered."""
    import torch
    c = Chain(*heads, 128, 5)
    (c.k if of_keys else c.v)[170, 0, 77] = value
    c.append()
    assert c.refused() == [1]
    assert c.attend() == INVALID_VALUE and bool(c.out.isnan().all()) and bool(c.lse.isnan().all())
    c.end[1] = 0
    assert c.attend() == 0
    rows = [tuple(t[c.at(r)][:0 if r == 1 else None] for t in c.cache) for r in range(3)]
    A.check_rows(c.q, c.out, c.lse, rows, c.scale)
    # read back, only its block differs from a number of fp32
    got = [torch.empty(300, heads[1], 128, device="cuda", dtype=torch.bfloat16) for _ in range(2)]
    slots = c.table.repeat_interleave(PAGE, 1)[:, :100] * PAGE + torch.arange(100, device="cuda") % PAGE
    c.m.idx_cache_gather_fp4(*c.cache, slots.flatten().int(), *got)
    x = got[0 if of_keys else 1][170, 0].float()
    # -7 * 2^40 is 3.5 units of 2^41, halfway between the codes 5 (for 3) and 6 (for 4): the even one, -8 * 2^40
    want = -8 * 2.0 ** 40 if value == -7 * 2.0 ** 40 else value
    assert bool(x[64:96].isnan().all() if not math.isfinite(value) else x[77] == want)
    assert not any(bool(t[torch.arange(300, device="cuda") != 170].isnan().any()) for t in got)


@pytest.mark.parametrize("heads", [(8, 2), (64, 1)])
def test_the_largest_that_is_answered(heads):
    """6 * 2^40 has the largest scale byte that attention takes."""
    c = Chain(*heads, 128, 6)
    c.v[170, 0, 77] = 6 * 2.0 ** 40
    c.append()
    assert c.refused() == [] and int(c.cache[3].max()) == MAX_SCALE_BYTE
    assert c.attend() == 0
    A.check_rows(c.q, c.out, c.lse, [tuple(t[c.at(r)] for t in c.cache) for r in range(3)], c.scale)


@pytest.mark.parametrize("heads", [(8, 2), (64, 1)])
@pytest.mark.parametrize("big,small,e,scale", [(113, 85, 40, -4), (-60, -60, -40, 100), (100, 70, 20, -90)])
def test_scores_at_the_ends_of_what_is_kept(heads, big, small, e, scale):
    """A head's largest element 2^big, times keys' 2^e, from 2^-100 to 2^153: keys that meet only the element 2^small.  All
    numbers are powers of two, so a score is exact up to the scale in units of log2 (half a step) and its product with the
    maximum (another): 2^-23 of it, and log2 and the sum of two weights below 2^-20 more."""
    import torch
    c = Chain(*heads, 128, 7)
    for t, fill in zip(c.cache, (0, 0, 0x22, 127)):
        t.fill_(fill)
    c.q.zero_()
    c.q[:, :, 0], c.q[:, :, 40] = 2.0 ** big, 2.0 ** small
    c.cache[1][..., 1] = 127 + e                      # of elements 32 .. 63
    c.cache[0][..., 20] = 6                           # element 40: 4; of position 1: 2
    pg, of = c.at(0)
    c.cache[0][:, 1, :, 20] = 4
    c.scale = 2.0 ** scale
    c.end.fill_(2)
    assert c.attend() == 0
    s = 2.0 ** (small + e + 2 + scale)
    want = s + math.log1p(math.exp(-s / 2))
    lim = 2.0 ** -23 * (1 + 2.0 ** -20) * s + 2.0 ** -20 + 2.0 ** -22 * want
    assert float((c.lse.double() - want).abs().max()) <= lim
    assert bool((c.out == 1).all())
