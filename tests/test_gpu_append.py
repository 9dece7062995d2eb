"""Writing a paged cache in 16 bits and in 4, and reading a 4-bit one back, against plain forms (tests/append_ref.py, where
the bounds are derived): types, head layouts, norms, rotations, strides, padding rows, bad rows, ties and specials of the
4-bit form, graphs, and what must stay as it was."""
import numpy as np
import pytest

from tests import append_ref as A

pytestmark = pytest.mark.gpu

PAGE = 64
INVALID_METADATA, INVALID_PAGE = 3, 4


def _dt(name):
    import torch
    return {"bf16": torch.bfloat16, "f16": torch.float16}[name]


def pool(pages, heads, width, dtype, layout, n=2):
    """n tensors [pages, 64, heads, width] full of noise: slot by slot, head by head, or together in one allocation."""
    import torch
    make = (lambda *s: torch.randint(0, 256, s, device="cuda", dtype=torch.uint8)) if dtype == torch.uint8 else \
        (lambda *s: torch.randn(*s, device="cuda").to(dtype))
    if layout == "slot":
        return [make(pages, PAGE, heads, width) for _ in range(n)]
    if layout == "head":
        return [make(pages, heads, PAGE, width).transpose(1, 2) for _ in range(n)]
    both = make(pages, n, PAGE, heads, width)
    return [both[:, i] for i in range(n)]


class Case:
    """Rows (request, position or -1) over a paged cache in 16 or 4 bits."""

    def __init__(self, rows, hq, hk, dim, dtype="bf16", fp4=False, layout="slot", norm="same", rot=0, first=0, pairs=False, seed=1,
                 mp=4, nr=3, values=True, q4=False, table=None, pages=None, fused=True, scale=1.0):
        import torch
        torch.manual_seed(seed)
        rng = np.random.default_rng(seed)
        R, T = len(rows), _dt(dtype)
        self.rows, self.fp4, self.q4, self.dim, self.hk, self.hq, self.T = rows, fp4, q4, dim, hk, hq, T
        self.np_ = pages or nr * mp + 2
        self.table_host = table if table is not None else rng.permutation(self.np_)[:nr * mp].reshape(nr, mp).astype(np.int32)
        i32 = lambda x: torch.tensor(np.asarray(x, dtype=np.int32).tolist(), dtype=torch.int32, device="cuda")
        self.table = torch.from_numpy(np.ascontiguousarray(self.table_host)).cuda()
        self.req, self.pos = i32([r[0] for r in rows]), i32([r[1] for r in rows])
        x = (torch.randn(R, hq + 2 * hk, dim, device="cuda") * torch.exp2(torch.randn(dim, device="cuda")) * scale).to(T)
        if not fused:
            x = x.transpose(0, 1).contiguous().transpose(0, 1)
        self.q, self.k, self.v = (x[:, :hq] if hq else None), x[:, hq:hq + hk], (x[:, hq + hk:] if values else None)
        w = lambda: (1 + 0.3 * torch.randn(dim, device="cuda"))
        self.qw = self.kw = None
        if norm:
            self.kw = w().to(T if norm == "same" else torch.float32)
            self.qw = w().to(self.kw.dtype) if hq else None
        self.rot, self.first, self.pairs, self.rope = rot, first, pairs, None
        if rot:
            P = mp * PAGE
            angle = torch.arange(P, dtype=torch.float64)[:, None] * 10000.0 ** (-torch.arange(rot // 2, dtype=torch.float64) / (rot // 2))
            self.rope = torch.stack([angle.cos(), angle.sin()], 1).float().cuda()
        if fp4:
            n = 2 if values else 1
            self.codes, self.scales = pool(self.np_, hk, dim // 2, torch.uint8, layout, n), pool(self.np_, hk, dim // 32, torch.uint8, layout, n)
            self.caches = self.codes + self.scales
        else:
            self.caches = pool(self.np_, hk, dim, T, layout, 2 if values else 1)
        self.before = [c.clone() for c in self.caches]
        self.out_q = self.out_q_scale = None
        if hq:
            self.out_q = torch.full((R, hq, dim // 2), 77, device="cuda", dtype=torch.uint8) if q4 else \
                torch.full((hq, R, dim), 7.0, device="cuda", dtype=T).transpose(0, 1)
            if q4:
                self.out_q_scale = torch.full((R, hq, dim // 32), 77, device="cuda", dtype=torch.uint8)
        self.status = torch.full((1,), 99, dtype=torch.int32, device="cuda")
        self.eps = 1e-5

    def places(self):
        if self.fp4:
            v = (self.codes[1], self.scales[1]) if len(self.codes) == 2 else (None, None)
            return (self.codes[0], self.scales[0], *v)
        return (self.caches[0], self.caches[1] if len(self.caches) == 2 else None)

    def more(self):
        kw = dict(q=self.q, out_q=self.out_q, q_weight=self.qw, k_weight=self.kw, eps=self.eps, rope=self.rope, rope_first=self.first,
                  rope_pairs=self.pairs)
        return dict(kw, out_q_scale=self.out_q_scale) if self.fp4 else kw

    def run(self, asynchronous=False):
        import torch
        import fp4_sparse_attention_tma_gb300 as m
        fn = getattr(m, "idx_cache_append" + ("_fp4" if self.fp4 else "") + ("_async" if asynchronous else ""))
        tail = (self.status,) if asynchronous else ()
        code = fn(self.k, self.v, self.table, self.req, self.pos, *self.places(), *tail, **self.more(), raise_on_error=False)
        torch.cuda.synchronize()
        return int(self.status.item()) if asynchronous and code == 0 else code

    def want(self):
        """Of the rows that are there: places, and queries and keys in 64 bits with their bounds."""
        there = np.array([i for i, r in enumerate(self.rows) if r[1] >= 0], dtype=np.int64)
        req, pos = np.array([self.rows[i][0] for i in there], dtype=np.int64), np.array([self.rows[i][1] for i in there], dtype=np.int64)
        page = self.table_host[req, pos // PAGE]
        turn = (None, None) if self.rope is None else tuple(self.rope.cpu().numpy()[pos].transpose(1, 0, 2))
        return there, page, pos % PAGE, turn

    def form(self, x, w, turn, f, **kw):
        return f(x, None if w is None else A.to64(w), self.eps, *turn, self.first, self.pairs, **kw)

    def check(self):
        import torch
        there, page, off, turn = self.want()
        u = A.U[str(self.T).replace("torch.", "")]
        sub = 2.0 ** -25 if self.T == torch.float16 else 2.0 ** -134

        def near16(got, x, w):
            y, bound = self.form(A.to64(x)[there], w, turn, A.turned64, four=False)
            err = np.abs(A.to64(got) - y)
            lim = u * np.abs(y) + bound * (1 + u) + sub
            assert (err <= lim).all(), (float((err - lim).max()), np.argwhere(err > lim)[:4])
            if w is None and turn[0] is None:
                assert torch.equal(got, x[there])

        def near4(idx, scale, x, w):
            y, bound = self.form(A.to64(x)[there], w, turn, A.turned64)
            A.check_codes(idx, scale, y, bound)
            i32, s32 = A.quantise(self.form(A.to64(x)[there], w, turn, A.turned32))   # rounding by rounding
            assert (scale == s32).all() and (A.values(idx, scale) == A.values(i32, s32)).all()

        if self.hq:
            if self.q4:
                near4(A.unpack(self.out_q.cpu().numpy())[there], self.out_q_scale.cpu().numpy()[there], self.q, self.qw)
            else:
                near16(self.out_q[there], self.q, self.qw)
            skipped = [i for i in range(len(self.rows)) if i not in set(there.tolist())]
            if skipped:
                assert bool((self.out_q[skipped] == (77 if self.q4 else 7)).all())
        pg, of = torch.from_numpy(page).long().cuda(), torch.from_numpy(off).cuda()
        for i, (x, w) in enumerate([(self.k, self.kw), (self.v, None)]):
            if x is None:
                continue
            t = turn if i == 0 else (None, None)
            if self.fp4:
                idx, scale = A.unpack(self.codes[i][pg, of].cpu().numpy()), self.scales[i][pg, of].cpu().numpy()
                if i == 0:
                    near4(idx, scale, x, w)
                else:
                    want, s = A.quantise(A.to64(x)[there])
                    assert (scale == s).all() and (A.values(idx, scale) == A.values(want, s)).all()
            elif i == 0:
                near16(self.caches[0][pg, of], x, w)
            else:
                assert torch.equal(self.caches[1][pg, of], x[there])
        for now, old in zip(self.caches, self.before):   # everything else as it was
            keep = old.clone()
            keep[pg, of] = now[pg, of]
            assert torch.equal(now, keep)


ROWS = [(0, 0), (2, 255), (1, 63), (0, 64), (0, -1), (1, 64), (2, 128), (0, 1), (1, 200)]
ROT = [(0, 0, False), ("all", 0, False), ("all", 0, True), (32, 8, False), (64, -64, True), (48, 16, False), (16, 40, True)]


@pytest.mark.parametrize("fp4", [False, True])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("rot", ROT)
def test_forms(fp4, dtype, dim, rot):
    n, first, pairs = rot
    n, first = (dim if n == "all" else n), (first if first >= 0 else dim + first)
    for i, (hq, hk, norm, layout) in enumerate([(4, 2, "same", "slot"), (7, 1, "f32", "head"), (0, 5, None, "joint"), (3, 3, "same", "joint")]):
        c = Case(ROWS, hq, hk, dim, dtype, fp4, layout, norm, n, first, pairs, seed=i + 1, fused=i % 2 == 0, values=i != 1)
        assert c.run(asynchronous=i % 2 == 1) == 0
        c.check()


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("heads", [(64, 8), (33, 11), (1, 1)])
def test_many_rows(dim, heads):
    """The kernel for many heads at once: rows in any order, some of them not there."""
    rng = np.random.default_rng(dim)
    n = 400
    rows = [(int(s) // (64 * PAGE), int(s) % (64 * PAGE)) for s in rng.permutation(3 * 64 * PAGE)[:n]]
    rows = [(r, -1 if i % 37 == 5 else p) for i, (r, p) in enumerate(rows)]
    for fp4 in (False, True):
        c = Case(rows, *heads, dim, "bf16", fp4, "slot", "same", dim, 0, False, mp=64)
        assert c.run() == 0
        c.check()


@pytest.mark.parametrize("n", [16384, 16385, 40000])
def test_tens_of_thousands_of_rows(n):
    """More rows than the table of slots holds: a bitmap, in several parts where the pool is large."""
    nr, mp = 5, 4000
    rng = np.random.default_rng(n)
    table = rng.permutation(nr * mp + 17)[:nr * mp].reshape(nr, mp).astype(np.int32)
    rows = [(int(s) // (mp * PAGE), int(s) % (mp * PAGE)) for s in rng.permutation(nr * mp * PAGE)[:n]]
    c = Case(rows, 0, 1, 64, "bf16", True, norm=None, table=table, pages=nr * mp + 17, nr=nr, mp=mp)
    assert c.run() == 0
    c.check()
    c.pos[n - 1], c.req[n - 1] = rows[7][1], rows[7][0]     # the last row names the slot of the eighth
    c.before = [x.clone() for x in c.caches]
    c.k.zero_()
    assert c.run() == INVALID_PAGE
    assert all(bool((a == b).all()) for a, b in zip(c.caches, c.before))


def test_no_rows():
    for fp4 in (False, True):
        c = Case([], 4, 2, 128, fp4=fp4)
        assert c.run() == 0 and c.run(asynchronous=True) == 0
        assert all(bool((a == b).all()) for a, b in zip(c.caches, c.before))


def test_queries_in_place():
    import torch
    c = Case(ROWS, 8, 2, 128, rot=128)
    keep = c.q.clone()
    c.out_q = c.q
    assert c.run() == 0
    got, c.q = c.out_q.clone(), keep
    c.out_q = got
    c.rows = [r for r in c.rows]
    there = [i for i, r in enumerate(c.rows) if r[1] >= 0]
    assert torch.equal(got[4], keep[4])          # the row that is not there
    c.out_q[4] = 7.0
    c.check()
    assert len(there) == 8


@pytest.mark.parametrize("fp4", [False, True])
@pytest.mark.parametrize("asynchronous", [False, True])
def test_bad_rows_change_nothing(fp4, asynchronous):
    import torch
    bad = [((0, 256), INVALID_METADATA), ((0, -2), INVALID_METADATA), ((3, 0), INVALID_METADATA), ((-1, 0), INVALID_METADATA),
           ((0, 64), INVALID_PAGE), ((1, 63), INVALID_PAGE)]
    for many in (1, 40):
        for (row, code) in bad:
            base = [(2, p) for p in range(many)] + [(1, 63)]
            c = Case(base + [row], 8, 2, 128, fp4=fp4, rot=64)
            if row == (0, 64):
                c.table[0, 1] = c.np_               # a page past the end
            assert c.run(asynchronous) == code, (row, many)
            assert all(torch.equal(a, b) for a, b in zip(c.caches, c.before))
            assert bool(c.out_q.isnan().all())
    # a page that two requests share: two rows with one slot; other slots of it are fine
    c = Case([(0, 5), (1, 5)], 4, 2, 128, fp4=fp4)
    c.table[1, 0] = c.table[0, 0]
    assert c.run(asynchronous) == INVALID_PAGE
    c = Case([(0, 5), (1, 6)], 4, 2, 128, fp4=fp4)
    c.table[1, 0] = c.table[0, 0]
    c.table_host[1, 0] = c.table_host[0, 0]
    assert c.run(asynchronous) == 0
    c.check()
    # a position that the angles do not reach
    c = Case([(0, 100)], 4, 2, 128, fp4=fp4, rot=64)
    c.rope = c.rope[:100].contiguous()
    assert c.run(asynchronous) == INVALID_METADATA
    # entries that no row asks for may be anything; so may the request of a row that is not there
    c = Case([(0, 5), (99, -1), (1, 70)], 4, 2, 128, fp4=fp4)
    c.table[2], c.table[0, 1:], c.table[1, 0] = -9, 1 << 30, -1
    assert c.run(asynchronous) == 0
    c.rows[1] = (0, -1)
    c.check()
    # queries in place keep their values, codes of queries become scales of 255
    c = Case([(0, 5), (0, 5)], 4, 2, 128, fp4=fp4)
    c.out_q = c.q
    keep = c.q.clone()
    assert c.run(asynchronous) == INVALID_PAGE and torch.equal(c.q, keep)
    if fp4:
        c = Case([(0, 5), (0, 5)], 4, 2, 128, fp4=True, q4=True)
        assert c.run(asynchronous) == INVALID_PAGE
        assert bool((c.out_q == 0).all()) and bool((c.out_q_scale == 255).all())


@pytest.mark.parametrize("dim", [64, 128, 256])
def test_queries_in_4_bits(dim):
    for hq, rot, pairs in [(64, dim, False), (5, 16, True), (1, 0, False)]:
        c = Case(ROWS, hq, 1, dim, fp4=True, q4=True, rot=rot, pairs=pairs, values=False)
        assert c.run() == 0
        c.check()


def specials(T):
    """Values [n, 32] of one block each: every border between codes and its neighbours, extremes, zeros."""
    import torch
    borders = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0], dtype=torch.float64)
    near = torch.cat([borders, borders * (1 + 2.0 ** -7), borders * (1 - 2.0 ** -7)])
    near = torch.cat([near, torch.tensor([0.0, -0.0, 4.0, 6.0, 0.5, 1.0, 3.0, -6.0])])
    top = 2 if T == torch.float16 else 30
    rows = [near * 2.0 ** e for e in (0, -3, top, -10)] + [-near * 2.0 ** e for e in (0, 5)]
    rows += [torch.zeros(32, dtype=torch.float64), -torch.zeros(32, dtype=torch.float64)]
    big = 60000.0 if T == torch.float16 else 3.0e38
    small = 2.0 ** -24 if T == torch.float16 else 2.0 ** -130
    rows += [torch.full((32,), big, dtype=torch.float64), torch.full((32,), small, dtype=torch.float64),
             torch.tensor([big] + [small] * 31, dtype=torch.float64), torch.tensor([6.0 + 2.0 ** -3] + [1.0] * 31, dtype=torch.float64),
             torch.tensor([3.0] + [0.1] * 31, dtype=torch.float64), torch.tensor([3.0 + 2.0 ** -6] + [0.1] * 31, dtype=torch.float64)]
    return torch.stack(rows).to(T)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_borders_of_the_4_bit_form(dtype):
    import torch
    T = _dt(dtype)
    x = specials(T)
    n = x.shape[0]
    x = torch.cat([x, x.flip(0)], 1)                        # two blocks a head
    c = Case([(0, i) for i in range(n)], 0, 1, 64, dtype, True, norm=None)
    c.k[:, 0], c.v[:, 0] = x.cuda(), x.flip(1).cuda()
    assert c.run() == 0
    c.check()
    assert len(set(c.scales[0][c.table[0, 0].long(), :n].flatten().tolist())) > 5


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_what_is_not_finite_becomes_a_scale_of_255(dtype):
    import torch
    import fp4_sparse_attention_tma_gb300 as m
    c = Case([(0, i) for i in range(6)], 0, 1, 64, dtype, True, norm=None)
    for i, (d, x) in enumerate([(0, float("nan")), (31, float("inf")), (32, -float("inf")), (63, float("nan"))]):
        c.v[i, 0, d] = x
    c.k[4, 0, 5] = float("nan")
    assert c.run() == 0
    page = int(c.table[0, 0])
    s = c.scales[1][page, :6, 0].tolist()
    assert [255 in r for r in s] == [True] * 4 + [False] * 2
    assert s[0][0] == 255 and s[0][1] != 255 and s[2][1] == 255 and s[3][1] == 255 and s[1][0] == 255
    assert c.scales[0][page, 4, 0, 0] == 255 and bool((c.codes[0][page, 4, 0, :16] == 0).all())
    ok = torch.empty(6, 1, 64, device="cuda", dtype=_dt(dtype))
    m.idx_cache_gather_fp4(c.codes[1], c.scales[1], None, None, (page * PAGE + torch.arange(6, device="cuda")).int(), ok, None)
    assert bool(ok[0, 0, :32].isnan().all()) and not bool(ok[0, 0, 32:].isnan().any()) and not bool(ok[4:].isnan().any())


def test_what_is_not_finite_goes_by_the_formula():
    """A norm over an infinity: the mean is infinite, every finite element 0, the infinite one NaN."""
    c = Case([(0, 0), (0, 1), (0, 2)], 1, 1, 64, "bf16", norm="same")
    c.q[0, 0, 3], c.q[1, 0, 4], c.q[2, 0] = float("inf"), float("nan"), 1e20
    assert c.run() == 0
    got = c.out_q[:, 0].float().cpu()
    assert got[0, 3].isnan() and (got[0, :3] == 0).all() and (got[0, 4:] == 0).all()
    assert got[1].isnan().all() and (got[2] == 0).all()      # (1e40 is beyond 32 bits)
    c = Case([(0, 0)], 1, 1, 64, "bf16", norm="same")
    c.q.zero_()
    c.eps = 0.0
    assert c.run() == 0
    assert c.out_q.isnan().all()                             # 0 / 0


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("layout", ["slot", "head", "joint"])
def test_gather(dtype, dim, layout):
    import torch
    import fp4_sparse_attention_tma_gb300 as m
    torch.manual_seed(dim)
    for hk, n in [(1, 1), (3, 70), (8, 5000), (5, 0)]:
        pages = 40
        codes, scales = pool(pages, hk, dim // 2, torch.uint8, layout), pool(pages, hk, dim // 32, torch.uint8, layout)
        for s in scales:
            s.copy_(torch.randint(100, 140, s.shape, device="cuda"))
        slots = torch.randint(-1, pages * PAGE, (n,), dtype=torch.int32, device="cuda")
        if n:
            slots[-1] = -1 if n > 1 else pages * PAGE - 1
        out = [torch.full((hk, n, dim), 7.0, device="cuda", dtype=_dt(dtype)).transpose(0, 1) for _ in range(2)]
        m.idx_cache_gather_fp4(codes[0], scales[0], codes[1], scales[1], slots, *out)
        at = slots.long().clamp(min=0)
        for c, s, o in zip(codes, scales, out):
            want = A.values(A.unpack(c[at // PAGE, at % PAGE].cpu().numpy()), s[at // PAGE, at % PAGE].cpu().numpy())
            want = np.where((slots >= 0).cpu().numpy()[:, None, None], want, 0.0)
            assert torch.equal(o.cpu(), torch.from_numpy(want).to(_dt(dtype)))
        alone = torch.empty(n, hk, dim, device="cuda", dtype=_dt(dtype))
        status = torch.full((1,), 9, dtype=torch.int32, device="cuda")
        m.idx_cache_gather_fp4_async(codes[1], scales[1], None, None, slots, alone, None, status)
        assert torch.equal(alone, out[1]) and int(status.item()) == 0
        for bad in (-2, pages * PAGE, 1 << 30):
            if n < 2:
                continue
            slots[n // 2] = bad
            assert m.idx_cache_gather_fp4(codes[0], scales[0], codes[1], scales[1], slots, *out, raise_on_error=False) == INVALID_PAGE
            assert bool(out[0][n // 2].isnan().all()) and bool(out[1][n // 2].isnan().all())
            alone[n // 2] = out[1][n // 2]
            assert torch.equal(alone.view(torch.int16), out[1].contiguous().view(torch.int16))


def test_gather_every_scale():
    """All scale bytes: subnormal results, overflow to infinity, NaN; rounded once."""
    import torch
    import fp4_sparse_attention_tma_gb300 as m
    codes = torch.arange(256, dtype=torch.uint8, device="cuda").view(1, 1, 1, 256)[..., :32].repeat(4, 64, 1, 1)
    codes[..., 16:] = torch.randint(0, 256, (4, 64, 1, 16), device="cuda", dtype=torch.uint8)
    scales = torch.arange(256, dtype=torch.uint8, device="cuda").view(4, 64, 1, 1).repeat(1, 1, 1, 2)
    for dtype in (torch.bfloat16, torch.float16):
        out = torch.empty(256, 1, 64, device="cuda", dtype=dtype)
        m.idx_cache_gather_fp4(codes, scales, None, None, torch.arange(256, dtype=torch.int32, device="cuda"), out, None)
        want = A.values(A.unpack(codes.view(256, 1, 32).cpu().numpy()), scales.view(256, 1, 2).cpu().numpy())
        want = torch.from_numpy(want).to(dtype)
        same = (out.cpu() == want) | (out.cpu().isnan() & want.isnan())
        assert bool(same.all()), torch.nonzero(~same)[:4]


def test_into_the_indexers_cache():
    """Keys and queries that this wrote, scored by the indexer: 64 query heads, one key of 128 dimensions."""
    import torch
    import fp4_sparse_attention_tma_gb300 as m
    n, mp = 700, 11
    c = Case([(0, i) for i in range(n)], 64, 1, 128, fp4=True, q4=True, values=False, rot=64, first=64, pairs=True, mp=mp, nr=1)
    c.scales[0].fill_(120)                                  # (the indexer looks at whole pages)
    c.before[1].fill_(120)
    assert c.run() == 0
    c.check()
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
    rows = 5
    q4, qs = c.out_q[-rows:].contiguous(), c.out_q_scale[-rows:].contiguous()
    weights = torch.randn(rows, 64, device="cuda")
    end = [n - rows + 1 + i for i in range(rows)]
    args = dict(q_fp4=q4, q_scale=qs, k_cache_fp4=c.codes[0].view(-1, 64, 64), k_scale=c.scales[0].view(-1, 64, 4), weights=weights,
                page_table=c.table, row_req=i32([0] * rows), row_start=i32([0] * rows), row_end=i32(end))
    scores = torch.empty(rows, mp * PAGE, device="cuda")
    m.idx_fp4_debug_scores(**args, out_scores=scores)
    q = A.values(A.unpack(q4.cpu().numpy()), qs.cpu().numpy())
    pos = np.arange(n)
    page = c.table_host[0, pos // PAGE]
    k = A.values(A.unpack(c.codes[0].cpu().numpy()[page, pos % PAGE, 0]), c.scales[0].cpu().numpy()[page, pos % PAGE, 0])
    dots = np.maximum(np.einsum("rhd,nd->rhn", q, k), 0) * A.to64(weights)[..., None]
    # 2^-24 for each of the products (exact up to the accumulation of 128 terms) and of the sums over 64 heads
    lim = (128 + 64 + 2) * 2.0 ** -23 * np.abs(dots).sum(1) + 128 * 2.0 ** -23 * np.einsum("rhd,nd->rn", np.abs(q) * np.abs(A.to64(weights))[..., None], np.abs(k))
    for r in range(rows):
        err = np.abs(scores[r, :end[r]].double().cpu().numpy() - dots[r].sum(0)[:end[r]])
        assert (err <= lim[r, :end[r]] + 1e-30).all()


def test_graph_and_streams():
    """Captured, replayed with other rows, and on a stream of its own."""
    import torch
    import fp4_sparse_attention_tma_gb300 as m
    c = Case([(0, 10), (1, 11)], 4, 2, 128, fp4=True, rot=128)
    side = torch.cuda.Stream()
    out = [torch.zeros(2, 2, 128, device="cuda", dtype=c.T) for _ in range(2)]
    slots = torch.zeros(2, dtype=torch.int32, device="cuda")
    c.run(asynchronous=True)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.stream(side), torch.cuda.graph(graph, stream=side):
        m.idx_cache_append_fp4_async(c.k, c.v, c.table, c.req, c.pos, *c.places(), c.status, **c.more())
        m.idx_cache_gather_fp4_async(c.codes[0], c.scales[0], c.codes[1], c.scales[1], slots, *out, c.status)
        with pytest.raises(m.IdxError):                     # the synchronous form is refused while capturing
            m.idx_cache_append_fp4(c.k, c.v, c.table, c.req, c.pos, *c.places(), **c.more())
    for rows in [[(0, 12), (2, 0)], [(1, 63), (1, 64)], [(2, 255), (0, -1)]]:
        c.rows = rows
        c.k.copy_(torch.randn_like(c.k))
        c.req.copy_(torch.tensor([r[0] for r in rows]))
        c.pos.copy_(torch.tensor([r[1] for r in rows]))
        slots.copy_(torch.where(c.pos >= 0, c.table[c.req.long(), c.pos.long().clamp(min=0) // PAGE] * PAGE + c.pos % PAGE, -1))
        c.out_q.fill_(7.0)
        c.before = [x.clone() for x in c.caches]
        graph.replay()
        torch.cuda.synchronize()
        assert int(c.status.item()) == 0
        c.check()
        at = slots.long()
        for i in range(2):
            want = A.values(A.unpack(c.codes[i][at // PAGE, at % PAGE].cpu().numpy()), c.scales[i][at // PAGE, at % PAGE].cpu().numpy())
            want[(at < 0).cpu().numpy()] = 0
            assert torch.equal(out[i].cpu(), torch.from_numpy(want).to(c.T))
    c2 = Case([(0, 10), (1, 11)], 4, 2, 128, rot=128)
    side.wait_stream(torch.cuda.current_stream())
    m.idx_cache_append(c2.k, c2.v, c2.table, c2.req, c2.pos, *c2.places(), **c2.more(), stream=side)
    torch.cuda.synchronize()
    c2.check()


def test_offsets_beyond_32_bits():
    """A pool of 2^31 elements and more: the last page."""
    import torch
    c = Case([(0, 70)], 0, 8, 256, norm=None, nr=1, mp=2)
    pages = (1 << 31) // (64 * 8 * 256) + 3
    big = torch.zeros(pages, PAGE, 8, 256, device="cuda", dtype=torch.bfloat16)
    c.caches[0] = big
    c.caches[1] = torch.zeros(pages, PAGE, 8, 256, device="cuda", dtype=torch.bfloat16)
    c.table_host[0, 1] = pages - 1
    c.table[0, 1] = pages - 1
    assert c.run() == 0
    assert torch.equal(c.caches[0][pages - 1, 6], c.k[0]) and torch.equal(c.caches[1][pages - 1, 6], c.v[0])
    assert int((c.caches[0] != 0).any(-1).sum()) == 8


@pytest.mark.parametrize("pages", [3, 40, 200, 17000])
@pytest.mark.parametrize("n", [2, 33, 190])
def test_slots_named_twice_in_pools_of_many_sizes(pages, n):
    """Found whatever finds them; slots that differ by a page, or by many, are not taken for one another."""
    import torch
    rng = np.random.default_rng(pages + n)
    mp = min(pages, 190)
    n = min(n, mp * PAGE)
    table = np.sort(rng.permutation(pages)[:mp]).reshape(1, mp).astype(np.int32)
    for step in (1, PAGE):                       # neighbours; the first slots of the pages, then the second ones
        at = [(i * step) % (mp * PAGE) + (i * step) // (mp * PAGE) for i in range(n)]
        c = Case([(0, x) for x in at], 0, 1, 64, "f16", True, norm=None, table=table, pages=pages, nr=1, mp=mp)
        assert c.run() == 0
        c.check()
        c.before = [x.clone() for x in c.caches]
        c.pos[0] = at[n - 1]
        c.k.zero_()
        assert c.run() == INVALID_PAGE
        assert all(bool((a == b).all()) for a, b in zip(c.caches, c.before))
