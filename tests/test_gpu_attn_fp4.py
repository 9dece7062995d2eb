"""Attention over a cache in 4 bits, paged and over lists of slots, against plain 64-bit attention (tests/attn4_ref.py,
where the bounds are derived): types, head layouts, lengths, windows, strides, scales of every size, what no row sees,
scales that are refused, streams, graphs, and the chain from writing the cache to reading it."""
import math

import numpy as np
import pytest

from tests import attn4_ref as A

pytestmark = pytest.mark.gpu

PAGE = 64
INVALID_ARGUMENT, INVALID_METADATA, INVALID_PAGE, INVALID_VALUE = 1, 3, 4, 10


def _dt(name):
    import torch
    return {"bf16": torch.bfloat16, "f16": torch.float16}[name]


def make_cache(pages, heads, dim, layout, seed, lo=122, hi=128):
    """(key codes, key scales, value codes, value scales): random codes, scale bytes lo .. hi - 1."""
    import torch
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    got = []
    for width, a, b in [(dim // 2, 0, 256), (dim // 32, lo, hi)] * 2:
        make = lambda *s: torch.randint(a, b, s, device="cuda", dtype=torch.uint8, generator=g)
        if layout == "slot":
            got.append(make(pages, PAGE, heads, width))
        elif layout == "head":
            got.append(make(pages, heads, PAGE, width).transpose(1, 2))
        else:                                       # every head's row inside a wider one
            pad = -(-width // 16) * 16 + 16 if width >= 16 else 4 * width
            got.append(make(pages, PAGE, heads, pad)[..., :width] if width >= 16 else make(pages, PAGE, heads, pad)[..., :width])
    return got


class Case:
    """A cache with requests of the given lengths, and rows (request, start, end)."""

    def __init__(self, lens, wins, hq, hk, dim, dtype="bf16", layout="slot", seed=1, q_strided=False, lo=122, hi=128):
        import torch
        rng = np.random.default_rng(seed)
        need = [-(-n // PAGE) for n in lens]
        self.np_ = max(1, sum(need)) + 2
        perm = rng.permutation(self.np_)
        self.mp = max(1, max(need))
        table = np.full((len(lens), self.mp), -1, dtype=np.int32)
        at = 0
        for i, n in enumerate(need):
            table[i, :n] = perm[at:at + n]
            at += n
        self.table = torch.from_numpy(table).cuda()
        self.cache = make_cache(self.np_, hk, dim, layout, seed, lo, hi)
        g = torch.Generator(device="cuda")
        g.manual_seed(seed + 1)
        R = len(wins)
        if q_strided:
            wide = torch.randn(R, hq + 2 * hk, dim, device="cuda", generator=g).to(_dt(dtype))
            self.q = wide[:, :hq]
            self.out = torch.full((hq, R, dim), 7.0, device="cuda", dtype=_dt(dtype)).transpose(0, 1)
        else:
            self.q = torch.randn(R, hq, dim, device="cuda", generator=g).to(_dt(dtype))
            self.out = torch.full((R, hq, dim), 7.0, device="cuda", dtype=_dt(dtype))
        i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
        self.wins = wins
        self.req, self.start, self.end = i32([w[0] for w in wins]), i32([w[1] for w in wins]), i32([w[2] for w in wins])
        self.scale = 1.0 / math.sqrt(dim)
        self.lse = torch.full((R, hq), 7.0, device="cuda")
        self.hq, self.hk, self.dim = hq, hk, dim

    def args(self):
        return (self.q, *self.cache, self.table, self.req, self.start, self.end, self.scale, self.out)

    def at(self, req, pos):
        import torch
        pos = torch.as_tensor(pos)
        return self.table.cpu()[req][pos // PAGE].long().cuda(), (pos % PAGE).cuda()

    def rows(self):
        import torch
        return [tuple(t[self.at(i, torch.arange(a, max(a, b)))] for t in self.cache) for i, a, b in self.wins]

    def check(self):
        A.check_rows(self.q, self.out, self.lse, self.rows(), self.scale)


def run_paged(c, **kw):
    import torch
    import fp4_sparse_attention_tma_gb300 as m
    code = m.idx_attn_paged_fp4(*c.args(), out_lse=c.lse, raise_on_error=False, **kw)
    torch.cuda.synchronize()
    return code


def run_slots(c, slots):
    import torch
    import fp4_sparse_attention_tma_gb300 as m
    code = m.idx_attn_selected_fp4(c.q, *c.cache, slots, c.scale, c.out, out_lse=c.lse, raise_on_error=False)
    torch.cuda.synchronize()
    return code


def check_slots(c, slots):
    rows = []
    for r in range(slots.shape[0]):
        s = slots[r][slots[r] >= 0].long()
        rows.append(tuple(t[s // PAGE, s % PAGE] for t in c.cache))
    A.check_rows(c.q, c.out, c.lse, rows, c.scale)


LENS = [1, 0, 15, 16, 17, 31, 32, 33, 63, 64, 65, 200, 1000]


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("heads", [(1, 1), (8, 8), (32, 8), (12, 4), (5, 1), (64, 1), (40, 2)])
def test_one_row(dtype, dim, heads):
    c = Case(LENS, [(i, 0, n) for i, n in enumerate(LENS)], *heads, dim, dtype)
    assert run_paged(c) == 0
    c.check()


@pytest.mark.parametrize("layout", ["slot", "head", "wide"])
@pytest.mark.parametrize("heads", [(4, 4), (16, 2), (64, 1), (9, 3)])
def test_rows_share_the_cache(layout, heads):
    """Several rows of a request, each seeing one position more, and sliding windows."""
    lens = [3, 70, 500, 1, 129]
    wins = []
    for i, n in enumerate(lens):
        for j in range(4):
            e = max(0, n - (3 - j))
            wins.append((i, max(0, e - (100 if i == 2 else 1 << 20)), e))
    for dim in (64, 128, 256):
        c = Case(lens, wins, *heads, dim, layout=layout, q_strided=True)
        assert run_paged(c) == 0
        c.check()


@pytest.mark.parametrize("heads", [(8, 2), (64, 1), (64, 2)])
def test_windows_of_every_offset(heads):
    """Starts and ends at every place of a subtile and page; empty windows between them; rows whose windows do not meet."""
    wins = [(0, a, b) for a, b in [(0, 0), (5, 5), (1, 2), (63, 65), (64, 64), (15, 16), (16, 33), (100, 300), (299, 300),
                                   (127, 129), (0, 300), (17, 17), (250, 251), (48, 64), (31, 33), (0, 32), (32, 64)]]
    c = Case([300], wins, *heads, 128)
    assert run_paged(c) == 0
    c.check()
    wins = [(0, 0, 10), (0, 200, 290), (0, 0, 0), (0, 130, 131), (0, 290, 300)]
    c = Case([300], wins, *heads, 128)
    c.table[0, 1] = -5                                  # under no window
    assert run_paged(c) == 0
    c.check()


@pytest.mark.parametrize("n_rows", [257, 700])
@pytest.mark.parametrize("heads,dim", [((6, 2), 64), ((64, 1), 128)])
def test_many_rows(n_rows, heads, dim):
    rng = np.random.default_rng(n_rows)
    lens = [int(x) for x in rng.integers(0, 90, 37)]
    wins = []
    for _ in range(n_rows):
        i = int(rng.integers(0, 37))
        a = int(rng.integers(0, lens[i] + 1))
        wins.append((i, a, int(rng.integers(a, lens[i] + 1))))
    c = Case(lens, wins, *heads, dim)
    assert run_paged(c) == 0
    c.check()


@pytest.mark.parametrize("heads,dim", [((32, 8), 128), ((64, 1), 128), ((16, 1), 64), ((8, 2), 256), ((64, 8), 128), ((24, 1), 128)])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_long(heads, dim, dtype):
    c = Case([20011, 9000], [(0, 0, 20011), (1, 0, 8999), (1, 0, 9000)], *heads, dim, dtype)
    assert run_paged(c) == 0
    c.check()


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("heads", [(1, 1), (32, 8), (64, 1), (14, 2)])
@pytest.mark.parametrize("n", [1, 17, 512])
def test_selected(dtype, dim, heads, n):
    for layout in ("slot", "head", "wide"):
        c, slots = slot_case(9, n, *heads, dim, dtype, layout)
        assert run_slots(c, slots) == 0
        check_slots(c, slots)


def slot_case(R, n, hq, hk, dim, dtype="bf16", layout="slot", seed=3, context=4096, holes=True, **kw):
    import torch
    c = Case([context], [(0, 0, 0)] * R, hq, hk, dim, dtype, layout, seed, **kw)
    rng = np.random.default_rng(seed)
    slots = np.full((R, n), -1, dtype=np.int32)
    for r in range(R):
        m = n if not holes else int(rng.integers(0, n + 1))
        if r == 0 and holes:
            m = 0
        at = rng.choice(n, m, replace=False) if r % 2 else np.arange(m)
        slots[r, at] = rng.choice(c.np_ * PAGE, m, replace=m > c.np_ * PAGE)
    return c, torch.from_numpy(slots).cuda()


@pytest.mark.parametrize("heads,n", [((64, 1), 130), ((8, 2), 65), ((64, 1), 1024), ((40, 2), 200)])
def test_selected_many_rows_and_duplicates(heads, n):
    c, slots = slot_case(1500 if n < 1000 else 200, n, *heads, 128)
    slots[5, :] = slots[5, 0]           # one slot many times (or none)
    assert run_slots(c, slots) == 0
    check_slots(c, slots)


# ------------------------------------------------------------------ scales ----

@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("heads", [(16, 2), (64, 1)])
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("span", [(0, 1), (167, 168), (0, 30), (90, 140), (127, 128), (20, 60)])
def test_scales_of_every_size(dtype, heads, dim, span):
    """Blocks far apart in scale; queries brought to the keys' size, so that the weights are not all on one position."""
    import torch
    lo, hi = span
    c = Case([300, 33], [(0, 0, 299), (0, 0, 300), (1, 0, 33)], *heads, dim, dtype, lo=lo, hi=hi)
    c.scale = 0.3 * 2.0 ** -(min(hi, 130) - 127) / dim if hi > 100 else 0.3 * 2.0 ** 100 / dim
    if dtype == "f16" and hi > 142:                       # values within fp16's range (keys beyond it)
        c.cache[3].fill_(130)
        c.scale = 0.3 * 2.0 ** -(hi - 128) / dim
    elif hi > 150:
        c.scale = 0.3 * 2.0 ** -(hi - 128) / dim
    assert run_paged(c) == 0
    c.check()
    c, slots = slot_case(5, 100, *heads, dim, dtype, lo=lo, hi=min(hi, 143) if dtype == "f16" and lo < 143 else hi)
    c.scale = 0.1 * 2.0 ** -(min(hi, 143) - 127) / dim if lo > 60 else 0.1 / dim
    if dtype == "f16" and lo >= 143:
        c.cache[3].fill_(127)
        c.scale = 0.1 * 2.0 ** -(hi - 128) / dim
    assert run_slots(c, slots) == 0
    check_slots(c, slots)


@pytest.mark.parametrize("heads", [(8, 1), (64, 1), (32, 2)])
@pytest.mark.parametrize("order", ["rising", "falling", "one"])
def test_values_whose_scale_changes_along_the_context(heads, order):
    """The values' reference follows them: from small to large, from large to small, one large position among small ones."""
    import torch
    n = 700
    c = Case([n], [(0, 0, n - 1), (0, 0, n)], *heads, 128)
    pg, of = c.at(0, torch.arange(n))
    step = torch.arange(n, device="cuda") // 16
    e = {"rising": 100 + step, "falling": 144 - step, "one": torch.where(torch.arange(n, device="cuda") == 333, 140, 115)}[order]
    c.cache[3][pg, of] = e.to(torch.uint8)[:, None, None]
    assert run_paged(c) == 0
    c.check()
    # channels of their own size, as a layer's loud channels: each keeps its precision
    c = Case([n], [(0, 0, n)], *heads, 128)
    c.cache[3][:] = torch.tensor([115, 120, 127, 132], dtype=torch.uint8, device="cuda")
    assert run_paged(c) == 0
    c.check()
    k, ks, v, vs = c.rows()[0]
    want, _, bo, _ = A.attend(c.q[0], A.values(k, ks), A.values(v, vs), c.scale, int(ks.max()), 0)
    for b in range(4):
        part = slice(32 * b, 32 * b + 32)
        err = (c.out[0, :, part].double() - want[:, part]).abs().max()
        assert float(err) <= 2.0 ** -8 * 6 * 2.0 ** ([115, 120, 127, 132][b] - 127)


@pytest.mark.parametrize("heads,rows", [((8, 1), 2), ((8, 4), 3), ((64, 1), 2), ((64, 1), 1)])
def test_what_no_row_sees(heads, rows):
    """Codes and scales (255 among them) outside the windows change nothing, bit for bit; inside they are refused."""
    import torch
    wins = [(0, 3, 98), (0, 3, 99), (0, 4, 98)][:rows]
    c = Case([100], wins, *heads, 128)
    out = []
    for k in range(2):
        hide = list(range(0, 3)) + list(range(max(w[2] for w in wins), 128))
        pg, of = c.at(0, hide)
        c.cache[1][pg, of] = 255 if k else 0
        c.cache[3][pg, of] = 255 if k else 7
        c.cache[0][pg, of] = torch.randint(0, 256, c.cache[0][pg, of].shape, device="cuda", dtype=torch.uint8)
        c.cache[2][pg, of] = torch.randint(0, 256, c.cache[2][pg, of].shape, device="cuda", dtype=torch.uint8)
        assert run_paged(c) == 0
        c.check()
        out.append((c.out.clone(), c.lse.clone()))
    assert torch.equal(out[0][0], out[1][0]) and torch.equal(out[0][1], out[1][1])
    for which in (1, 3):
        for bad in (168, 255):
            for pos in (3, 97):
                pg, of = c.at(0, [pos])
                keep = c.cache[which].clone()
                c.cache[which][pg, of, -1, -1] = bad
                assert run_paged(c) == INVALID_VALUE
                assert bool(c.out.isnan().all()) and bool(c.lse.isnan().all())
                c.cache[which].copy_(keep)
    assert run_paged(c) == 0 and torch.equal(c.out, out[1][0])


@pytest.mark.parametrize("heads", [(8, 2), (64, 1)])
def test_selected_ignores_what_is_not_listed(heads):
    import torch
    c, slots = slot_case(6, 40, *heads, 128)
    on = torch.zeros(c.np_ * PAGE, dtype=torch.bool, device="cuda")
    on[slots[slots >= 0].long()] = True
    off = (~on).view(c.np_, PAGE)
    c.cache[1][off], c.cache[3][off] = 255, 255
    assert run_slots(c, slots) == 0
    check_slots(c, slots)
    s = int(slots[slots >= 0][3])
    c.cache[3][s // PAGE, s % PAGE, 0, 1] = 168
    assert run_slots(c, slots) == INVALID_VALUE
    assert bool(c.out.isnan().all())
    c.cache[3][s // PAGE, s % PAGE, 0, 1] = 127
    for bad in (-2, c.np_ * PAGE, 1 << 30):
        slots[4, 7] = bad
        assert run_slots(c, slots) == INVALID_PAGE
        assert bool(c.out.isnan().all()) and bool(c.lse.isnan().all())


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("heads", [(8, 2), (64, 1)])
def test_queries_of_every_size(dtype, heads):
    """Tiny, huge and mixed queries: scores up to 2^31 and beyond, weights on one position, none lost."""
    import torch
    sizes = [2.0 ** -100, 2.0 ** -20, 1.0, 2.0 ** 12, 2.0 ** 60] if dtype == "bf16" else [2.0 ** -14, 1.0, 2.0 ** 12]
    for size in sizes:
        c = Case([500], [(0, 0, 500)], *heads, 128, dtype)
        c.q = (c.q.double() * size).to(c.q.dtype)
        c.q[:, :, 5] = c.q[:, :, 5] * 2.0 ** -6
        assert run_paged(c) == 0
        c.check()
    c = Case([500], [(0, 0, 500)], *heads, 128, dtype)
    c.q.zero_()
    assert run_paged(c) == 0
    c.check()                                                 # all weights alike


@pytest.mark.parametrize("heads", [(8, 2), (64, 1)])
def test_queries_that_are_not_finite(heads):
    import torch
    c = Case([100], [(0, 0, 100), (0, 0, 99)], *heads, 128)
    keep = c.q.clone()
    assert run_paged(c) == 0
    want = c.out.clone()
    for bad in (float("nan"), float("inf")):
        c.q.copy_(keep)
        c.q[0, 1, 7] = bad
        assert run_paged(c) == 0
        assert bool(c.out[0, 1].isnan().all())
        ok = torch.ones_like(c.lse, dtype=torch.bool)
        ok[0, 1] = False
        assert torch.equal(c.out[ok], want[ok])


def test_long_tail_under_one_heavy_position():
    """One position with nearly all the weight, and many small ones together as large: the tail is not lost."""
    import torch
    n = 60000
    for heads in ((8, 1), (64, 1)):
        for dtype in ("bf16", "f16"):
            c = Case([n], [(0, 0, n)], *heads, 128, dtype)
            c.cache[0].zero_()
            pg, of = c.at(0, [17])
            c.cache[0][pg, of] = 0x22                         # 1.0 everywhere
            c.cache[1].fill_(127)
            c.q.fill_(11.0 * math.sqrt(128) / 128)            # a score of 11 there, 0 elsewhere: weights e^11 = 59874 and 1
            c.cache[2].fill_(0x22)
            c.cache[2][pg, of] = 0xAA                         # -1
            c.cache[3].fill_(127)
            assert run_paged(c) == 0
            c.check()


# ------------------------------------------------- calls, streams and graphs ----

def test_bad_metadata_and_pages():
    import torch
    for heads in ((8, 2), (64, 1)):
        for change, code in [(("req", 0, 2), INVALID_METADATA), (("start", 1, -1), INVALID_METADATA), (("end", 2, 321), INVALID_METADATA),
                             (("start", 2, 301), INVALID_METADATA), (("table", (0, 2), -1), INVALID_PAGE),
                             (("table", (0, 0), 1 << 20), INVALID_PAGE)]:
            c = Case([300, 100], [(0, 0, 300), (1, 0, 99), (0, 100, 300)], *heads, 128)
            getattr(c, change[0])[change[1]] = change[2]
            assert run_paged(c) == code, change
            assert bool(c.out.isnan().all()) and bool(c.lse.isnan().all())


def test_no_rows_and_no_positions():
    import torch
    import fp4_sparse_attention_tma_gb300 as m
    c = Case([100], [(0, 5, 5), (0, 0, 0)], 8, 2, 128)
    assert run_paged(c) == 0
    assert bool((c.out == 0).all()) and bool(torch.isneginf(c.lse).all())
    e = torch.empty(0, dtype=torch.int32, device="cuda")
    assert m.idx_attn_paged_fp4(c.q[:0], *c.cache, c.table, e, e, e, 0.1, c.out[:0]) == 0


def space(c, slots=None):
    import torch
    import fp4_sparse_attention_tma_gb300 as m
    R = c.q.shape[0]
    n = m.idx_attn_paged_fp4_scratch_bytes(R, c.hq, c.hk, c.dim, *c.table.shape) if slots is None else \
        m.idx_attn_selected_fp4_scratch_bytes(R, c.hq, c.hk, c.dim, slots.shape[1])
    return torch.full((n,), 0xA5, dtype=torch.uint8, device="cuda"), torch.full((1,), -7, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("heads", [(16, 4), (64, 1)])
def test_stream_ordered_and_graphs(heads):
    """The same bits on any stream, again, and captured; two graphs replayed at once with workspaces of their own."""
    import torch
    import fp4_sparse_attention_tma_gb300 as m
    c = Case([3000, 65, 700], [(0, 0, 3000), (1, 0, 65), (2, 0, 699), (2, 0, 700)], *heads, 128)
    c2, slots = slot_case(40, 300, *heads, 128)
    assert run_paged(c) == 0 and run_slots(c2, slots) == 0
    want, wl, want2 = c.out.clone(), c.lse.clone(), c2.out.clone()
    ws, st = space(c)
    ws2, st2 = space(c2, slots)
    call = lambda: m.idx_attn_paged_fp4_async(*c.args(), ws, st, out_lse=c.lse)
    call2 = lambda: m.idx_attn_selected_fp4_async(c2.q, *c2.cache, slots, c2.scale, c2.out, ws2, st2, out_lse=c2.lse)
    short = torch.empty(ws.numel() - 256, dtype=torch.uint8, device="cuda")
    assert m.idx_attn_paged_fp4_async(*c.args(), short[:256], st, raise_on_error=False) == INVALID_ARGUMENT
    graphs = []
    call(), call2()
    torch.cuda.synchronize()
    for f in (call, call2):
        s, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
        with torch.cuda.stream(s), torch.cuda.graph(g, stream=s):
            f()
        graphs.append((s, g))
    for k in range(4):
        c.out.fill_(3.0), c2.out.fill_(3.0), st.fill_(-7), st2.fill_(-7)
        torch.cuda.synchronize()
        for s, g in graphs:
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        assert int(st.item()) == 0 and int(st2.item()) == 0
        assert torch.equal(c.out, want) and torch.equal(c.lse, wl) and torch.equal(c2.out, want2)
    c.end.copy_(torch.tensor([2000, 0, 650, 651], dtype=torch.int32))
    c.wins = [(0, 0, 2000), (1, 0, 0), (2, 0, 650), (2, 0, 651)]
    graphs[0][1].replay()
    torch.cuda.synchronize()
    c.check()
    side = torch.cuda.Stream()
    c2.out.fill_(3.0)
    torch.cuda.synchronize()
    m.idx_attn_selected_fp4_async(c2.q, *c2.cache, slots, c2.scale, c2.out, ws2, st2, stream=side)
    torch.cuda.synchronize()
    assert torch.equal(c2.out, want2)


def test_offsets_beyond_32_bits():
    """Caches of more than 2^32 bytes, and of more than 2^32 pieces of 16 bytes (by their strides)."""
    import torch
    import fp4_sparse_attention_tma_gb300 as m
    for far in (False, True):
        pages, hk, dim = 4200, 16, 256
        each = (16 << 20) + 4096 if far else (1 << 20)       # bytes from a page to the next
        codes = torch.empty(pages * each, dtype=torch.uint8, device="cuda")
        used = [pages - 1, 0, pages - 2, 4097]
        k = codes.as_strided((pages, PAGE, hk, dim // 2), (each, hk * dim // 2, dim // 2, 1))
        v = codes.as_strided((pages, PAGE, hk, dim // 2), (each, hk * dim // 2, dim // 2, 1), 262144)
        ks, vs = (torch.randint(120, 128, (pages, PAGE, hk, dim // 32), dtype=torch.uint8, device="cuda") for _ in range(2))
        for t in (k, v):
            for p in used:
                t[p] = torch.randint(0, 256, t[p].shape, dtype=torch.uint8, device="cuda")
        assert codes.numel() > (2 ** 36 if far else 2 ** 32)
        table = torch.tensor([used], dtype=torch.int32, device="cuda")
        q = torch.randn(1, 16, dim, device="cuda").to(torch.bfloat16)
        i32 = lambda x: torch.tensor([x], dtype=torch.int32, device="cuda")
        out, lse = torch.empty_like(q), torch.empty(1, 16, device="cuda")
        m.idx_attn_paged_fp4(q, k, ks, v, vs, table, i32(0), i32(0), i32(250), 0.06, out, out_lse=lse)
        pos = torch.arange(250, device="cuda")
        pg, of = table[0][pos // PAGE].long(), pos % PAGE
        rows = [tuple(t[pg, of] for t in (k, ks, v, vs))]
        A.check_rows(q, out, lse, rows, 0.06)
        slots = (pg * PAGE + of).to(torch.int32)[None].contiguous()
        m.idx_attn_selected_fp4(q, k, ks, v, vs, slots, 0.06, out, out_lse=lse)
        A.check_rows(q, out, lse, rows, 0.06)
        del codes, k, v
        torch.cuda.empty_cache()


@pytest.mark.parametrize("hq,hk,dim", [(8, 2, 128), (64, 1, 128), (4, 4, 64)])
def test_from_writing_to_attending(hq, hk, dim):
    """Prompts written, then tokens one by one with attention after each, paged and over all slots: the same numbers."""
    import torch
    import fp4_sparse_attention_tma_gb300 as m
    torch.manual_seed(hq)
    lens, mp, P = [70, 3, 129], 4, 256
    table = torch.randperm(3 * mp + 2, device="cuda")[:3 * mp].view(3, mp).to(torch.int32)
    cache = [torch.full((3 * mp + 2, PAGE, hk, w), 255, dtype=torch.uint8, device="cuda") for w in (dim // 2, dim // 32) * 2]
    angle = torch.arange(P, dtype=torch.float64)[:, None] * 10000.0 ** (-torch.arange(dim // 2) / (dim / 2))
    rope = torch.stack([angle.cos(), angle.sin()], 1).float().cuda()
    w = [(1 + 0.1 * torch.randn(dim, device="cuda")).bfloat16() for _ in range(2)]
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
    step = lambda req, pos: (torch.randn(len(req), hq + 2 * hk, dim, device="cuda").bfloat16(), i32(req), i32(pos))

    def write(x, req, pos):
        q = x[:, :hq]
        m.idx_cache_append_fp4(x[:, hq:hq + hk], x[:, hq + hk:], table, req, pos, *cache, q=q, out_q=q, q_weight=w[0], k_weight=w[1],
                               eps=1e-6, rope=rope)
        return q

    write(*step([i for i, n in enumerate(lens) for _ in range(n)], [p for n in lens for p in range(n)]))
    for t in range(3):
        x, req, pos = step([0, 1, 2], lens)
        q = write(x, req, pos)
        lens = [n + 1 for n in lens]
        out, lse = torch.empty(3, hq, dim, device="cuda", dtype=torch.bfloat16), torch.empty(3, hq, device="cuda")
        m.idx_attn_paged_fp4(q, *cache, table, req, i32([0, 0, 0]), i32(lens), dim ** -0.5, out, out_lse=lse)
        rows, slots = [], torch.full((3, 200), -1, dtype=torch.int32, device="cuda")
        for i, n in enumerate(lens):
            p = torch.arange(n, device="cuda")
            pg, of = table[i][p // PAGE].long(), p % PAGE
            rows.append(tuple(c[pg, of] for c in cache))
            slots[i, :n] = (pg * PAGE + of).to(torch.int32)
        A.check_rows(q, out, lse, rows, dim ** -0.5)
        m.idx_attn_selected_fp4(q, *cache, slots, dim ** -0.5, out, out_lse=lse)
        A.check_rows(q, out, lse, rows, dim ** -0.5)


@pytest.mark.parametrize("heads", [(64, 2), (16, 1)])
def test_offsets_beyond_32_bits_many_heads(heads):
    """A cache of more than 2^32 bytes where its tiles are fed to the tensor memory's products."""
    import torch
    import fp4_sparse_attention_tma_gb300 as m
    (hq, hk), pages, dim, each, rows = heads, 4300, 128, 1 << 20, 2
    codes = torch.empty(pages * each, dtype=torch.uint8, device="cuda")
    assert codes.numel() > 2 ** 32
    used = [pages - 1, 0, pages - 2, 4097]
    k = codes.as_strided((pages, PAGE, hk, dim // 2), (each, hk * dim // 2, dim // 2, 1))
    v = codes.as_strided((pages, PAGE, hk, dim // 2), (each, hk * dim // 2, dim // 2, 1), 262144)
    ks, vs = (torch.randint(120, 128, (pages, PAGE, hk, dim // 32), dtype=torch.uint8, device="cuda") for _ in range(2))
    for t in (k, v):
        for p in used:
            t[p] = torch.randint(0, 256, t[p].shape, dtype=torch.uint8, device="cuda")
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
    table, pos = i32([used]), torch.arange(250, device="cuda")
    q = torch.randn(rows, hq, dim, device="cuda").to(torch.bfloat16)
    out, lse = torch.empty_like(q), torch.empty(rows, hq, device="cuda")
    m.idx_attn_paged_fp4(q, k, ks, v, vs, table, i32([0, 0]), i32([0, 3]), i32([250, 251]), 0.06, out, out_lse=lse)
    at = lambda pos: tuple(t[table[0][pos // PAGE].long(), pos % PAGE] for t in (k, ks, v, vs))
    A.check_rows(q, out, lse, [at(pos), at(pos[2:] + 1)], 0.06)
    slots = (table[0][pos // PAGE].long() * PAGE + pos % PAGE).to(torch.int32)[None].expand(rows, -1).contiguous()
    m.idx_attn_selected_fp4(q, k, ks, v, vs, slots, 0.06, out, out_lse=lse)
    A.check_rows(q, out, lse, [at(pos)] * rows, 0.06)


@pytest.mark.parametrize("heads", [(8, 2), (64, 1)])
def test_no_rows(heads):
    """No rows, and no pages either: nothing to do, and no error."""
    import torch
    import fp4_sparse_attention_tma_gb300 as m
    hq, hk = heads
    z = lambda *s, dtype=torch.uint8: torch.zeros(*s, dtype=dtype, device="cuda")
    i32 = lambda *s: z(*s, dtype=torch.int32)
    for pages in (0, 2):
        cache = [z(pages, PAGE, hk, w) for w in (64, 4, 64, 4)]
        q, out = (z(0, hq, 128, dtype=torch.bfloat16) for _ in range(2))
        lse = z(0, hq, dtype=torch.float32)
        m.idx_attn_paged_fp4(q, *cache, i32(1, 2), i32(0), i32(0), i32(0), 0.1, out, out_lse=lse)
        m.idx_attn_selected_fp4(q, *cache, i32(0, 8), 0.1, out, out_lse=lse)
        st = i32(1) + 7
        ws = z(m.idx_attn_selected_fp4_scratch_bytes(0, hq, hk, 128, 8))
        m.idx_attn_selected_fp4_async(q, *cache, i32(0, 8), 0.1, out, ws, st)
        assert int(st.item()) == 0
