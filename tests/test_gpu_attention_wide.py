"""Attention with more than 16 query heads per key-value head at head dimension 128: two rows
of a request share their tiles, one row's heads stand twice.  Windows that meet in every way,
values that only one of the two may notice, lists with holes, far offsets.  Bounds as derived
in tests/attn_ref.py."""
import numpy as np
import pytest

from tests import attn_ref as A
from tests import test_gpu_attention as B

pytestmark = pytest.mark.gpu

PAGE = 64
# windows of two rows of one request of 700 positions
PAIRS = [((0, 699), (0, 700)), ((0, 700), (0, 699)),            # one position more, or fewer
         ((0, 100), (200, 600)), ((200, 600), (0, 100)),        # apart, either first
         ((0, 400), (150, 700)), ((150, 700), (0, 400)),        # sliding
         ((0, 700), (300, 320)), ((300, 320), (0, 700)),        # one inside the other
         ((128, 256), (256, 384)), ((127, 129), (128, 130)),    # at a tile's edge
         ((0, 0), (0, 700)), ((0, 700), (9, 9)), ((0, 0), (700, 700)),   # one or both see nothing
         ((0, 1), (699, 700)), ((5, 6), (5, 6)), ((64, 640), (64, 640)),
         ((100, 700), (0, 700)), ((1, 513), (129, 385))]


@pytest.mark.parametrize("heads", [(64, 1), (17, 1), (66, 2), (128, 2), (65, 1), (130, 1)])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_two_rows_of_a_request(heads, dtype):
    """Every pair of windows, each in a request of its own, with a third row behind some of them."""
    wins = []
    for i, (x, y) in enumerate(PAIRS):
        wins += [(i, *x), (i, *y)]
        if i % 3 == 0:
            wins.append((i, 33, 690))       # pairs begin at odd rows from here
    c = B.Case([700] * len(PAIRS), wins, *heads, 128, dtype, q_strided=heads == (64, 1))
    assert B.run_paged(c) == 0
    c.check()


@pytest.mark.parametrize("pair", PAIRS)
def test_a_pair_alone(pair):
    """One pair: its tiles are divided among many workers, and joined."""
    c = B.Case([700], [(0, *pair[0]), (0, *pair[1])], 64, 1, 128)
    assert B.run_paged(c) == 0
    c.check()


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("pair", [((0, 699), (0, 700)), ((0, 700), (0, 600)), ((0, 400), (150, 700)), ((150, 700), (0, 400)),
                                  ((0, 700), (300, 320)), ((0, 100), (200, 600))])
def test_what_one_row_sees_never_reaches_the_other(pair, bad):
    """What only the first row sees, then what only the second sees, turns bad in keys and values."""
    import torch
    for copies in (1, 60):       # one pair over many workers; many pairs, several a worker
        wins = [(i, *w) for i in range(copies) for w in pair]
        c = B.Case([700] * copies, wins, 64, 1, 128)
        t = c.table.cpu()
        assert B.run_paged(c) == 0
        want = c.out.clone()
        k0, v0 = c.k.clone(), c.v.clone()
        for j in (0, 1):
            mine, other = pair[j], pair[1 - j]
            only = [x for x in range(*mine) if not other[0] <= x < other[1]]
            if not only:
                continue
            pos = torch.tensor(only)
            for i in range(copies):
                page, off = t[i][pos // PAGE].long().cuda(), (pos % PAGE).cuda()
                c.k[page, off] = bad
                c.v[page, off] = bad
            assert B.run_paged(c) == 0
            rows = range(1 - j, 2 * copies, 2)
            assert bool((c.out[rows] == want[rows]).all())
            assert not bool(c.out[range(j, 2 * copies, 2)].isfinite().all())
            c.k.copy_(k0)
            c.v.copy_(v0)


@pytest.mark.parametrize("heads", [(64, 1), (96, 1)])
def test_many_rows(heads):
    """More rows than are kept at hand; requests in any order, empty rows among them."""
    rng = np.random.default_rng(heads[0])
    lens = [int(x) for x in rng.integers(0, 400, 41)]
    wins = []
    for _ in range(650):
        i = int(rng.integers(0, 41))
        for _ in range(int(rng.integers(1, 4))):
            a = int(rng.integers(0, lens[i] + 1))
            wins.append((i, a, int(rng.integers(a, lens[i] + 1))))
    c = B.Case(lens, wins, *heads, 128)
    assert B.run_paged(c) == 0
    c.check()


@pytest.mark.parametrize("heads", [(64, 1), (40, 2), (80, 1)])
def test_weights_of_pairs(heads):
    import torch
    wins = [(i, *w) for i, p in enumerate(PAIRS) for w in p]
    c = B.Case([700] * len(PAIRS), wins, *heads, 128)
    wout = torch.full((len(PAIRS), c.mp * PAGE), 7.0, device="cuda")
    assert B.run_paged(c, weight_out=wout) == 0
    c.check()
    tot, bound = B._want_weights(c, None)
    assert bool(((wout.double() - tot).abs() <= bound).all())


@pytest.mark.parametrize("lens,wins", [([30000], [(0, 0, 29999), (0, 0, 30000)]),
                                       ([9000, 5, 14001], [(0, 200, 8999), (0, 0, 9000), (1, 0, 5), (2, 0, 14001), (2, 7000, 14000)]),
                                       ([40000], [(0, 17, 39990)])])
def test_long(lens, wins):
    for dtype in ("bf16", "f16"):
        c = B.Case(lens, wins, 64, 1, 128, dtype)
        assert B.run_paged(c) == 0
        c.check()


@pytest.mark.parametrize("n", [1, 63, 64, 65, 128, 129, 500, 1024])
def test_selected_holes(n):
    """Lists whose first or second halves of a tile, whole tiles, or everything, are missing."""
    import torch
    import fp4_sparse_attention_tma_gb300 as m
    c, slots = B._slot_case(12, n, 64, 1, 128, holes=False)
    at = torch.arange(n, device="cuda")
    slots[1, at % 128 < 64] = -1
    slots[2, at % 128 >= 64] = -1
    slots[3, at < n - 1] = -1
    slots[4, 1:] = -1
    slots[5, at // 128 % 2 == 0] = -1
    slots[6, :] = -1
    slots[7, at % 32 != 5] = -1
    slots[8, at // 128 % 2 == 1] = -1
    slots[10, at % 3 == 0] = -1
    m.idx_attn_selected(c.q, c.k, c.v, slots, c.scale, c.out, out_lse=c.lse)
    torch.cuda.synchronize()
    B._check_selected(c, slots)


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_selected_ignores_what_is_not_listed(bad):
    import torch
    import fp4_sparse_attention_tma_gb300 as m
    c, slots = B._slot_case(200, 300, 64, 1, 128)
    on = torch.zeros(c.np_ * PAGE, dtype=torch.bool, device="cuda")
    on[slots[slots >= 0].long()] = True
    on[:4000:3] = False                     # some that were listed are not any more
    slots[~on[slots.clamp(min=0).long()]] = -1
    off = (~on).view(c.np_, PAGE)
    c.k[off] = bad
    c.v[off] = bad
    m.idx_attn_selected(c.q, c.k, c.v, slots, c.scale, c.out, out_lse=c.lse)
    torch.cuda.synchronize()
    B._check_selected(c, slots)


@pytest.mark.parametrize("span", ["beyond 32 bits", "beyond 64 GB"])
def test_far_offsets(span):
    """Pages far apart in one allocation, of which a few are written and read."""
    import torch
    import fp4_sparse_attention_tma_gb300 as m
    dim, pages = 128, 5
    step = (2 ** 32 // 2 // 4 if span == "beyond 32 bits" else 2 ** 33) + 8 * 129    # elements between pages
    if torch.cuda.mem_get_info()[0] < 2 * 4 * step + (8 << 30):
        pytest.skip("not enough free memory")
    flat = torch.empty(4 * step + 2 * PAGE * dim, device="cuda", dtype=torch.bfloat16)
    k = flat.as_strided((pages, PAGE, 1, dim), (step, dim, dim, 1))
    v = flat.as_strided((pages, PAGE, 1, dim), (step, dim, dim, 1), PAGE * dim)
    g = torch.Generator(device="cuda")
    g.manual_seed(11)
    for p in range(pages):
        k[p] = torch.randn(PAGE, 1, dim, device="cuda", generator=g).to(torch.bfloat16)
        v[p] = torch.randn(PAGE, 1, dim, device="cuda", generator=g).to(torch.bfloat16)
    q = torch.randn(2, 64, dim, device="cuda", generator=g).to(torch.bfloat16)
    order = [4, 0, 3, 1, 2]
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
    out, lse = torch.empty_like(q), torch.empty(2, 64, device="cuda")
    m.idx_attn_paged(q, k, v, i32([order]), i32([0, 0]), i32([0, 3]), i32([319, 320]), 0.09, out, out_lse=lse)
    pos = torch.arange(320)
    pg, off = torch.tensor(order)[pos // PAGE].cuda(), (pos % PAGE).cuda()
    kk = torch.stack([k[int(a), int(b)] for a, b in zip(pg, off)])
    vv = torch.stack([v[int(a), int(b)] for a, b in zip(pg, off)])
    rows = [(kk[:319], vv[:319]), (kk[3:], vv[3:])]
    A.check_rows(q, out, lse, rows, 0.09)
    slots = (pg * PAGE + off).to(torch.int32)
    lists = torch.full((2, 320), -1, dtype=torch.int32, device="cuda")
    lists[0, :319] = slots[:319]
    lists[1, 3:] = slots[3:]
    out.zero_()
    m.idx_attn_selected(q, k, v, lists, 0.09, out, out_lse=lse)
    A.check_rows(q, out, lse, rows, 0.09)


def test_device_errors_fail_closed():
    import torch
    import fp4_sparse_attention_tma_gb300 as m
    for wins in ([(0, 0, 300), (0, 0, 300), (1, 0, 100)], [(0, 0, 300), (1, 0, 100)]):
        c = B.Case([300, 100], wins, 64, 1, 128)
        good = c.table.clone()
        for bad in (-1, 10 ** 6):
            c.table[0, 2] = bad
            assert B.run_paged(c) == B.INVALID_PAGE
            assert bool(c.out.isnan().all()) and bool(c.lse.isnan().all())
            c.table.copy_(good)
        assert B.run_paged(c) == 0
        c.check()
        c.end[0] = 6 * PAGE + 1
        assert B.run_paged(c) == B.INVALID_METADATA
        assert bool(c.out.isnan().all())
    c, slots = B._slot_case(5, 200, 64, 1, 128)
    slots[3, 150] = c.np_ * PAGE
    assert m.idx_attn_selected(c.q, c.k, c.v, slots, c.scale, c.out, out_lse=c.lse, raise_on_error=False) == B.INVALID_PAGE
    torch.cuda.synchronize()
    assert bool(c.out.isnan().all()) and bool(c.lse.isnan().all())


def test_same_bits_again_and_in_a_graph():
    import torch
    import fp4_sparse_attention_tma_gb300 as m
    wins = [(i, *w) for i, p in enumerate(PAIRS) for w in p]
    c = B.Case([700] * len(PAIRS), wins, 64, 1, 128)
    w = torch.zeros(len(PAIRS), c.mp * PAGE, device="cuda")
    assert B.run_paged(c, weight_out=w) == 0
    out, lse, w0 = c.out.clone(), c.lse.clone(), w.clone()
    ws, st = B._space(c, with_weights=True)
    s, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.stream(s):
        with torch.cuda.graph(g, stream=s):
            assert m.idx_attn_paged_async(*c.args(), ws, st, out_lse=c.lse, weight_out=w) == 0
    for _ in range(3):
        c.out.fill_(3.0)
        g.replay()
        torch.cuda.synchronize()
        assert int(st.item()) == 0
        assert bool((c.out == out).all()) and bool((c.lse == lse).all()) and bool((w == w0).all())


@pytest.mark.parametrize("heads", [(8, 8), (4, 1), (32, 8), (16, 1), (10, 2)])
@pytest.mark.parametrize("dtype,layout", [("bf16", "slot"), ("f16", "joint"), ("bf16", "head")])
def test_few_heads_over_long_contexts(heads, dtype, layout):
    """Up to 16 query heads per key-value head, one and two rows a request, where the context is long
    enough for the wide tiles; three rows, where it is not the context that decides."""
    lens = [3000, 2200, 1, 0, 130]
    wins = [(0, 0, 2999), (0, 7, 3000), (1, 1000, 2199), (1, 0, 900), (2, 0, 1), (2, 0, 0), (3, 0, 0), (3, 0, 0), (4, 0, 129),
            (4, 0, 130)]
    for w in (wins, wins[::2], wins + [(0, 100, 2500), (1, 2000, 2200), (4, 64, 128), (2, 0, 1), (3, 0, 0)]):
        c = B.Case(lens, w, *heads, 128, dtype, layout, q_strided=True)
        assert B.run_paged(c) == 0
        c.check()


@pytest.mark.parametrize("heads", [(8, 2), (16, 1), (3, 3)])
def test_weights_of_few_heads_over_long_contexts(heads):
    import torch
    wins = [(0, 0, 2500), (1, 100, 2100), (0, 2400, 2500), (2, 0, 0), (1, 0, 50)]
    c = B.Case([2500, 2100, 5], wins, *heads, 128)
    win = torch.rand(3, c.mp * PAGE, device="cuda")
    wout = torch.full_like(win, 7.0)
    assert B.run_paged(c, weight_in=win, weight_out=wout) == 0
    c.check()
    tot, bound = B._want_weights(c, win)
    assert bool(((wout.double() - tot).abs() <= bound).all())


@pytest.mark.parametrize("heads", [(8, 2), (16, 1), (32, 8), (2, 2)])
@pytest.mark.parametrize("n", [1023, 1024, 1100])
def test_selected_few_heads_of_long_lists(heads, n):
    import torch
    import fp4_sparse_attention_tma_gb300 as m
    for dtype, layout in (("bf16", "slot"), ("f16", "head"), ("bf16", "joint")):
        c, slots = B._slot_case(40, n, *heads, 128, dtype, layout)
        slots[3, :700] = -1
        m.idx_attn_selected(c.q, c.k, c.v, slots, c.scale, c.out, out_lse=c.lse)
        torch.cuda.synchronize()
        B._check_selected(c, slots)


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("heads", [(8, 1), (32, 8)])
def test_few_heads_and_what_one_row_sees(bad, heads):
    import torch
    c = B.Case([2500, 2400], [(0, 3, 2498), (0, 3, 2500), (1, 200, 2000), (1, 100, 1900)], *heads, 128)
    t = c.table.cpu()
    assert B.run_paged(c) == 0
    want = c.out.clone()
    for req, row, only in ((0, 1, range(2498, 2500)), (1, 2, range(1900, 2000)), (1, 3, range(100, 200)), (0, None, range(0, 3))):
        k0, v0 = c.k.clone(), c.v.clone()
        pos = torch.tensor(list(only))
        page, off = t[req][pos // PAGE].long().cuda(), (pos % PAGE).cuda()
        c.k[page, off] = bad
        c.v[page, off] = bad
        assert B.run_paged(c) == 0
        for r in range(4):
            if r == row:
                assert not bool(c.out[r].isfinite().all())
            else:
                assert bool((c.out[r] == want[r]).all())
        c.k.copy_(k0)
        c.v.copy_(v0)


def test_no_rows_over_a_wide_table():
    import torch
    import fp4_sparse_attention_tma_gb300 as m
    c = B.Case([3000], [(0, 0, 3000)], 8, 2, 128)
    win = torch.rand(1, c.mp * PAGE, device="cuda")
    wout = torch.zeros_like(win)
    e = torch.empty(0, dtype=torch.int32, device="cuda")
    assert m.idx_attn_paged(c.q[:0], c.k, c.v, c.table, e, e, e, 0.1, c.out[:0], weight_in=win, weight_out=wout) == 0
    torch.cuda.synchronize()
    assert bool((wout == win).all())
    for rows in (0, 1, 5):
        assert m.idx_attn_paged_scratch_bytes(rows, 8, 2, 128, 2, 1000) > 0


@pytest.mark.parametrize("requests", [3, 200])
def test_short_windows_under_a_wide_table(requests):
    """Few units, and many, where the table alone says that rows may be long."""
    wins = [(i, 2300 - 7 * i, 2400 - 5 * i) for i in range(requests)]
    c = B.Case([2400] * requests, wins, 16, 4, 128, "f16")
    assert B.run_paged(c) == 0
    c.check()


@pytest.mark.parametrize("heads", [(8, 8), (32, 8), (64, 1), (96, 2)])
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_workspace_does_not_depend_on_the_context(heads, dim):
    """One workspace serves every width of the page table and every length of the lists."""
    import fp4_sparse_attention_tma_gb300 as m
    for rows, reqs in ((1, 1), (7, 3), (64, 32), (3000, 1500)):
        assert len({m.idx_attn_paged_scratch_bytes(rows, *heads, dim, reqs, mp) for mp in (1, 31, 32, 5000)}) == 1
        assert len({m.idx_attn_selected_scratch_bytes(rows, *heads, dim, n) for n in (1, 512, 1024, 100000)}) == 1
    c = B.Case([2500, 100], [(0, 0, 2500), (1, 0, 100), (0, 5, 2400)], *heads, dim)
    ws, st = B._space(c)
    assert m.idx_attn_paged_async(*c.args(), ws, st, out_lse=c.lse) == 0
    import torch
    torch.cuda.synchronize()
    assert int(st.item()) == 0
    c.check()
