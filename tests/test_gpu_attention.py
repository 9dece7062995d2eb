"""Attention over the paged cache and over selected slots against plain 64-bit attention
(tests/attn_ref.py, where the bounds are derived): types, head layouts, lengths from none to
thousands, windows, strides, masked infinities and NaN, offsets beyond 32 bits, streams and
graphs, accumulated weights, and what the calls refuse."""
import math

import numpy as np
import pytest

from tests import attn_ref as A

pytestmark = pytest.mark.gpu

PAGE = 64
UNSUPPORTED, INVALID_ARGUMENT, INVALID_METADATA, INVALID_PAGE = 2, 1, 3, 4


def _dt(name):
    import torch
    return {"bf16": torch.bfloat16, "f16": torch.float16}[name]


def make_cache(pages, heads, dim, dtype, layout, seed):
    import torch
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    r = lambda *s: torch.randn(*s, device="cuda", dtype=dtype, generator=g)
    if layout == "slot":
        return r(pages, PAGE, heads, dim), r(pages, PAGE, heads, dim)
    if layout == "head":
        return r(pages, heads, PAGE, dim).transpose(1, 2), r(pages, heads, PAGE, dim).transpose(1, 2)
    both = r(pages, 2, PAGE, heads, dim)
    return both[:, 0], both[:, 1]


class Case:
    """A cache with requests of the given lengths, and rows (request, start, end)."""

    def __init__(self, lens, wins, hq, hk, dim, dtype="bf16", layout="slot", seed=1, q_strided=False):
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
        self.k, self.v = make_cache(self.np_, hk, dim, _dt(dtype), layout, seed)
        g = torch.Generator(device="cuda")
        g.manual_seed(seed + 1)
        R = len(wins)
        if q_strided:   # the queries of a fused projection, the output transposed
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
        return (self.q, self.k, self.v, self.table, self.req, self.start, self.end, self.scale, self.out)

    def rows(self):
        import torch
        t = self.table.cpu()
        got = []
        for i, a, b in self.wins:
            pos = torch.arange(a, max(a, b))
            page = t[i][pos // PAGE].long().cuda()
            got.append((self.k[page, (pos % PAGE).cuda()], self.v[page, (pos % PAGE).cuda()]))
        return got

    def check(self):
        A.check_rows(self.q, self.out, self.lse, self.rows(), self.scale)


def run_paged(c, **kw):
    import torch
    import fp4_sparse_attention_tma_gb300 as m
    code = m.idx_attn_paged(*c.args(), out_lse=c.lse, raise_on_error=False, **kw)
    torch.cuda.synchronize()
    return code


LENS = [1, 0, 15, 16, 17, 63, 64, 65, 200, 1000]


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("heads", [(1, 1), (8, 8), (32, 8), (12, 4), (5, 1), (64, 1), (40, 2)])
def test_paged_one_row(dtype, dim, heads):
    c = Case(LENS, [(i, 0, n) for i, n in enumerate(LENS)], *heads, dim, dtype)
    assert run_paged(c) == 0
    c.check()


@pytest.mark.parametrize("layout", ["slot", "head", "joint"])
@pytest.mark.parametrize("heads", [(4, 4), (16, 2), (64, 1)])
def test_paged_rows_share_the_cache(layout, heads):
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


def test_paged_windows_of_every_offset():
    """Starts and ends at every place of a subtile and page; empty windows between them."""
    wins = [(0, a, b) for a, b in [(0, 0), (5, 5), (1, 2), (63, 65), (64, 64), (15, 16), (16, 33), (100, 300), (299, 300),
                                   (127, 129), (0, 300), (17, 17), (250, 251), (48, 64)]]
    c = Case([300], wins, 8, 2, 128)
    assert run_paged(c) == 0
    c.check()


@pytest.mark.parametrize("n_rows", [257, 700])
def test_paged_many_rows(n_rows):
    """More rows than the threads that look them over at once; requests in any order."""
    rng = np.random.default_rng(n_rows)
    lens = [int(x) for x in rng.integers(0, 90, 37)]
    wins = []
    for _ in range(n_rows):
        i = int(rng.integers(0, 37))
        a = int(rng.integers(0, lens[i] + 1))
        wins.append((i, a, int(rng.integers(a, lens[i] + 1))))
    c = Case(lens, wins, 6, 2, 64)
    assert run_paged(c) == 0
    c.check()


@pytest.mark.parametrize("heads,dim", [((32, 8), 128), ((64, 1), 128), ((16, 1), 64), ((8, 2), 256)])
def test_paged_long(heads, dim):
    c = Case([20011, 9000], [(0, 0, 20011), (1, 0, 8999), (1, 0, 9000)], *heads, dim, "f16")
    assert run_paged(c) == 0
    c.check()


def test_paged_offsets_beyond_32_bits():
    import torch
    import fp4_sparse_attention_tma_gb300 as m
    pages, hk, dim = 33000, 8, 128           # 2.2e9 elements in each cache
    k = torch.empty(pages, PAGE, hk, dim, device="cuda", dtype=torch.bfloat16)
    v = torch.empty_like(k)
    assert k.numel() > 2 ** 31
    used = [32999, 0, 32998, 32768]
    for p in used:
        k[p].normal_()
        v[p].normal_()
    table = torch.tensor([used], dtype=torch.int32, device="cuda")
    q = torch.randn(1, 16, dim, device="cuda").to(torch.bfloat16)
    i32 = lambda x: torch.tensor([x], dtype=torch.int32, device="cuda")
    out, lse = torch.empty_like(q), torch.empty(1, 16, device="cuda")
    m.idx_attn_paged(q, k, v, table, i32(0), i32(0), i32(250), 0.09, out, out_lse=lse)
    pos = torch.arange(250)
    pg = table.cpu()[0][pos // PAGE].long().cuda()
    A.check_rows(q, out, lse, [(k[pg, (pos % PAGE).cuda()], v[pg, (pos % PAGE).cuda()])], 0.09)
    slots = (pg * PAGE + (pos % PAGE).cuda()).to(torch.int32)[None].contiguous()
    out2 = torch.empty_like(q)
    m.idx_attn_selected(q, k, v, slots, 0.09, out2, out_lse=lse)
    A.check_rows(q, out2, lse, [(k[pg, (pos % PAGE).cuda()], v[pg, (pos % PAGE).cuda()])], 0.09)


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("heads", [(8, 1), (8, 4)])
def test_paged_masked_values_never_reach_a_row(bad, heads):
    """Keys and values outside the rows' windows hold NaN or infinities: behind the end, before
    the start, and where another row of the same group sees one of them."""
    lens = [100]
    c = Case(lens, [(0, 3, 98), (0, 3, 99), (0, 4, 98)], *heads, 128)
    t = c.table.cpu()[0]
    for pos in list(range(0, 3)) + list(range(99, 128)):
        c.k[int(t[pos // PAGE]), pos % PAGE] = bad
        c.v[int(t[pos // PAGE]), pos % PAGE] = bad
    assert run_paged(c) == 0
    c.check()
    # position 98 is row 1's alone: only it may notice
    c.v[int(t[1]), 98 - 64] = bad
    want = c.out.clone()
    assert run_paged(c) == 0
    assert bool((c.out[0] == want[0]).all()) and bool((c.out[2] == want[2]).all())
    assert not bool(c.out[1].isfinite().any())
    # and position 3 is not row 2's
    c.v[int(t[1]), 98 - 64] = 0.0
    c.k[int(t[0]), 3] = float("nan")
    assert run_paged(c) == 0
    assert bool((c.out[2] == want[2]).all())
    assert bool(c.out[0].isnan().all()) and bool(c.out[1].isnan().all())


def test_paged_scores_of_minus_infinity():
    """A visible key of -infinity has weight 0; a row of nothing else is NaN, as in the formula."""
    import torch
    c = Case([40, 40], [(0, 0, 40), (1, 0, 40)], 4, 1, 64)
    t = c.table.cpu()
    c.q.fill_(1.0)
    c.k[int(t[0][0]), 7] = -float("inf")
    c.k[int(t[1][0])] = -float("inf")
    assert run_paged(c) == 0
    k, v = c.rows()[0]
    on = torch.arange(40, device="cuda") != 7
    want, _, _, bo, _, _ = A.attend(c.q[0], k[on], v[on], c.scale)
    assert bool(((c.out[0].double() - want).abs() <= bo).all())
    assert bool(c.out[1].isnan().all()) and bool(torch.isneginf(c.lse[1]).all())


def _weights_case(hq=8, hk=2, dim=128):
    lens = [300, 1, 0, 77]
    # request 0's rows do not follow one another
    wins = [(0, 0, 299), (1, 0, 1), (0, 10, 300), (3, 5, 77), (3, 0, 0), (2, 0, 0), (0, 64, 128)]
    return Case(lens, wins, hq, hk, dim)


def _want_weights(c, win):
    import torch
    tot = torch.zeros(c.table.shape[0], c.mp * PAGE, dtype=torch.float64, device="cuda")
    err = torch.zeros_like(tot)
    for r, ((i, a, b), (k, v)) in enumerate(zip(c.wins, c.rows())):
        if b <= a:
            continue
        _, _, p, _, _, ep = A.attend(c.q[r], k, v, c.scale)
        tot[i, a:b] += p.sum(0)
        err[i, a:b] += (p * ep[:, None]).sum(0)
    if win is not None:
        tot = tot + win.double()
    return tot, err + 2.0 ** -22 * tot.abs() + 1e-30


@pytest.mark.parametrize("heads,dim", [((8, 2), 128), ((64, 1), 128), ((3, 3), 64), ((8, 1), 256)])
@pytest.mark.parametrize("mode", ["none", "apart", "in_place"])
def test_paged_weights(heads, dim, mode):
    import torch
    c = _weights_case(*heads, dim)
    g = torch.Generator(device="cuda")
    g.manual_seed(5)
    win = None if mode == "none" else torch.rand(4, c.mp * PAGE, device="cuda", generator=g) * 3
    base = None if win is None else win.clone()
    wout = win if mode == "in_place" else torch.full((4, c.mp * PAGE), 7.0, device="cuda")
    assert run_paged(c, weight_in=win, weight_out=wout) == 0
    c.check()
    tot, bound = _want_weights(c, base)
    assert bool(((wout.double() - tot).abs() <= bound).all()), float(((wout.double() - tot).abs() - bound).max())
    if mode == "none":
        assert bool((wout[2] == 0).all())


def test_paged_weights_without_rows():
    import torch
    import fp4_sparse_attention_tma_gb300 as m
    c = Case([100], [(0, 0, 100)], 4, 2, 64)
    win = torch.rand(1, c.mp * PAGE, device="cuda")
    wout = torch.zeros_like(win)
    e = torch.empty(0, dtype=torch.int32, device="cuda")
    m.idx_attn_paged(c.q[:0], c.k, c.v, c.table, e, e, e, 0.1, c.out[:0], weight_in=win, weight_out=wout)
    torch.cuda.synchronize()
    assert bool((wout == win).all())


def test_same_bits_again_and_on_another_stream():
    import torch
    import fp4_sparse_attention_tma_gb300 as m
    c = Case([5000, 2000, 31], [(0, 0, 5000), (1, 0, 1999), (1, 0, 2000), (2, 0, 31)], 16, 2, 128)
    w = torch.zeros(3, c.mp * PAGE, device="cuda")
    assert run_paged(c, weight_out=w) == 0
    out, lse, w0 = c.out.clone(), c.lse.clone(), w.clone()
    s = torch.cuda.Stream()
    for k in range(3):
        c.out.fill_(3.0)
        torch.cuda.synchronize()
        with torch.cuda.stream(s if k else torch.cuda.current_stream()):
            m.idx_attn_paged(*c.args(), out_lse=c.lse, weight_out=w, stream=s if k == 2 else None)
        torch.cuda.synchronize()
        assert bool((c.out == out).all()) and bool((c.lse == lse).all()) and bool((w == w0).all())


def _space(c, with_weights=False, slots=None):
    import torch
    import fp4_sparse_attention_tma_gb300 as m
    R = c.q.shape[0]
    n = m.idx_attn_paged_scratch_bytes(R, c.hq, c.hk, c.dim, *c.table.shape, with_weights=with_weights) if slots is None else \
        m.idx_attn_selected_scratch_bytes(R, c.hq, c.hk, c.dim, slots.shape[1])
    # garbage in the workspace must not matter
    return torch.full((n,), 0xA5, dtype=torch.uint8, device="cuda"), torch.full((1,), -7, dtype=torch.int32, device="cuda")


def test_stream_ordered_and_graph():
    import torch
    import fp4_sparse_attention_tma_gb300 as m
    c = Case([3000, 65, 700], [(0, 0, 3000), (1, 0, 65), (2, 0, 699), (2, 0, 700)], 16, 4, 128)
    w = torch.zeros(3, c.mp * PAGE, device="cuda")
    assert run_paged(c, weight_out=w) == 0
    want, wl, ww = c.out.clone(), c.lse.clone(), w.clone()
    ws, st = _space(c, with_weights=True)
    call = lambda: m.idx_attn_paged_async(*c.args(), ws, st, out_lse=c.lse, weight_out=w)
    c.out.fill_(3.0)
    assert call() == 0
    torch.cuda.synchronize()
    assert int(st.item()) == 0 and bool((c.out == want).all()) and bool((w == ww).all())
    s, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.stream(s):
        with torch.cuda.graph(g, stream=s):
            assert call() == 0
    for k in range(2):
        if k:   # new windows in the same buffers
            c.end.copy_(torch.tensor([2000, 0, 650, 651], dtype=torch.int32))
            c.wins = [(0, 0, 2000), (1, 0, 0), (2, 0, 650), (2, 0, 651)]
        c.out.fill_(3.0)
        st.fill_(-7)
        g.replay()
        torch.cuda.synchronize()
        assert int(st.item()) == 0
        if k == 0:
            assert bool((c.out == want).all()) and bool((c.lse == wl).all())
        c.check()


# ------------------------------------------------------------- selected ----

def _slot_case(R, n, hq, hk, dim, dtype="bf16", layout="slot", seed=3, context=4096, holes=True):
    import torch
    c = Case([context], [(0, 0, 0)] * R, hq, hk, dim, dtype, layout, seed)
    rng = np.random.default_rng(seed)
    slots = np.full((R, n), -1, dtype=np.int32)
    for r in range(R):
        m = n if not holes else int(rng.integers(0, n + 1))
        if r == 0 and holes:
            m = 0
        at = rng.choice(n, m, replace=False) if r % 2 else np.arange(m)
        slots[r, at] = rng.choice(c.np_ * PAGE, m, replace=m > c.np_ * PAGE)
    return c, torch.from_numpy(slots).cuda()


def _check_selected(c, slots):
    rows = []
    for r in range(slots.shape[0]):
        s = slots[r][slots[r] >= 0].long()
        rows.append((c.k[s // PAGE, s % PAGE], c.v[s // PAGE, s % PAGE]))
    A.check_rows(c.q, c.out, c.lse, rows, c.scale)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("heads", [(1, 1), (32, 8), (64, 1), (14, 2)])
@pytest.mark.parametrize("n", [1, 17, 512])
def test_selected(dtype, dim, heads, n):
    import torch
    import fp4_sparse_attention_tma_gb300 as m
    for layout in ("slot", "head", "joint"):
        c, slots = _slot_case(9, n, *heads, dim, dtype, layout)
        assert m.idx_attn_selected(c.q, c.k, c.v, slots, c.scale, c.out, out_lse=c.lse) == 0
        torch.cuda.synchronize()
        _check_selected(c, slots)


def test_selected_many_rows_and_duplicates():
    import torch
    import fp4_sparse_attention_tma_gb300 as m
    c, slots = _slot_case(1500, 130, 64, 1, 128, holes=True)
    slots[5, :] = slots[5, 0]           # one slot many times (or none)
    m.idx_attn_selected(c.q, c.k, c.v, slots, c.scale, c.out, out_lse=c.lse)
    torch.cuda.synchronize()
    _check_selected(c, slots)


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_selected_ignores_what_is_not_listed(bad):
    import torch
    import fp4_sparse_attention_tma_gb300 as m
    c, slots = _slot_case(6, 40, 8, 2, 128)
    on = torch.zeros(c.np_ * PAGE, dtype=torch.bool, device="cuda")
    on[slots[slots >= 0].long()] = True
    off = (~on).view(c.np_, PAGE)
    c.k[off] = bad
    c.v[off] = bad
    m.idx_attn_selected(c.q, c.k, c.v, slots, c.scale, c.out, out_lse=c.lse)
    torch.cuda.synchronize()
    _check_selected(c, slots)


def test_selected_of_the_indexer_equals_paged_over_the_same_positions():
    """The TopK's physical slots feed the sparse attention; a row no longer than topk lists its
    whole window, where both forms compute the same sums."""
    import torch
    import fp4_sparse_attention_tma_gb300 as m
    from fp4_sparse_attention_tma_gb300 import inputs
    from tests import helpers as H
    p = inputs.make_problem(5, [2000, 400], [[(0, 2000), (0, 500)], [(0, 399), (0, 400)]], topk=512)
    d = H.to_device(p)
    phys = torch.zeros((p.rows, 512), dtype=torch.int32, device="cuda")
    m.idx_topk_fp4_prefill(**d, topk=512, out_phys_slot=phys)
    k, v = make_cache(p.num_pages, 1, 128, torch.bfloat16, "slot", 9)
    q = torch.randn(p.rows, 64, 128, device="cuda").to(torch.bfloat16)
    out, lse = torch.empty_like(q), torch.empty(p.rows, 64, device="cuda")
    m.idx_attn_selected(q, k, v, phys, 0.088, out, out_lse=lse)
    rows = []
    for r in range(p.rows):
        s = phys[r][phys[r] >= 0].long()
        rows.append((k[s // PAGE, s % PAGE], v[s // PAGE, s % PAGE]))
    A.check_rows(q, out, lse, rows, 0.088)
    out2, lse2 = torch.empty_like(q), torch.empty_like(lse)
    m.idx_attn_paged(q, k, v, d["page_table"], d["row_req"], d["row_start"], d["row_end"], 0.088, out2, out_lse=lse2)
    for r in range(1, p.rows):
        want, _, _, bo, _, _ = A.attend(q[r], *rows[r], 0.088)
        assert bool(((out2[r].double() - want).abs() <= bo).all())


# -------------------------------------------------------------- refusals ----

def test_device_errors_fail_closed():
    import torch
    import fp4_sparse_attention_tma_gb300 as m
    base = lambda: Case([300, 100], [(0, 0, 300), (1, 0, 100)], 8, 2, 128)
    for name, value, code in [("req", [0, 2], INVALID_METADATA), ("req", [-1, 1], INVALID_METADATA),
                              ("start", [-1, 0], INVALID_METADATA), ("start", [0, 101], INVALID_METADATA),
                              ("end", [300, 5 * 64 + 1], INVALID_METADATA)]:
        c = base()
        getattr(c, name).copy_(torch.tensor(value, dtype=torch.int32))
        w = torch.zeros(2, c.mp * PAGE, device="cuda")
        keep = torch.ones(2, c.mp * PAGE, device="cuda")
        assert run_paged(c, weight_out=w) == code
        assert bool(c.out.isnan().all()) and bool(c.lse.isnan().all()) and bool(w.isnan().all())
        assert run_paged(c, weight_in=keep, weight_out=keep) == code
        assert bool((keep == 1).all())
    for bad in (-1, 10 ** 6):
        c = base()
        c.table[0, 2] = bad
        ws, st = _space(c)
        assert m.idx_attn_paged_async(*c.args(), ws, st, out_lse=c.lse) == 0
        torch.cuda.synchronize()
        assert int(st.item()) == INVALID_PAGE and bool(c.out.isnan().all())
        c.table[0, 2] = 0
        assert m.idx_attn_paged_async(*c.args(), ws, st, out_lse=c.lse) == 0
        torch.cuda.synchronize()
        assert int(st.item()) == 0
        c.check()
    c = base()
    c.table[1, 2:] = 10 ** 6      # under no window: never read
    assert run_paged(c) == 0
    for low in (True, False):
        c, slots = _slot_case(4, 40, 8, 2, 64, holes=False)
        slots[2, 33] = -2 if low else c.np_ * PAGE
        assert m.idx_attn_selected(c.q, c.k, c.v, slots, c.scale, c.out, out_lse=c.lse, raise_on_error=False) == INVALID_PAGE
        torch.cuda.synchronize()
        assert bool(c.out.isnan().all()) and bool(c.lse.isnan().all())


def test_refused_arguments():
    """Refused on the host, with nothing enqueued and the outputs untouched."""
    import torch
    import fp4_sparse_attention_tma_gb300 as m
    c = Case([300], [(0, 0, 300)], 8, 2, 128)
    ok = dict(q=c.q, k_cache=c.k, v_cache=c.v, page_table=c.table, row_req=c.req, row_start=c.start, row_end=c.end,
              scale=c.scale, out=c.out, out_lse=c.lse)

    def refused(code=INVALID_ARGUMENT, **kw):
        got = m.idx_attn_paged(**{**ok, **kw}, raise_on_error=False)
        torch.cuda.synchronize()
        assert got == code, (kw.keys(), got)
        assert bool((c.out == 7).all()) and bool((c.lse == 7).all())

    z = lambda *s, dt=torch.bfloat16: torch.zeros(*s, dtype=dt, device="cuda")
    refused(q=c.q.float())
    refused(q=c.q.half())                                        # another type than the cache's
    refused(v_cache=c.v[:, :, :1])
    refused(k_cache=c.k.cpu())
    refused(q=z(1, 7, 128), out=z(1, 7, 128))                    # 7 query heads over 2
    refused(out=z(1, 8, 64))
    refused(out=c.q)                                             # over an input
    refused(out=z(1, 1, 128).expand(1, 8, 128))                  # heads on one address
    refused(q=z(1 * 8 * 128 + 8)[4:4 + 1024].view(1, 8, 128))    # 8-byte aligned
    refused(q=z(8 * 132)[:8 * 132].view(1, 8, 132)[:, :, :128])  # stride of 132
    refused(scale=0.0)
    refused(scale=float("nan"))
    refused(scale=float("inf"))
    refused(scale=-1.0)
    refused(row_end=c.end.long())
    refused(row_req=z(2, dt=torch.int32))
    refused(page_table=z(1, 2 * c.mp, dt=torch.int32)[:, ::2])
    refused(out_lse=z(1, 7, dt=torch.float32))
    refused(weight_in=z(1, c.mp * PAGE, dt=torch.float32))       # no place for the total
    refused(weight_out=z(1, c.mp * PAGE - 1, dt=torch.float32))
    refused(UNSUPPORTED, q=z(1, 8, 96), out=z(1, 8, 96), k_cache=z(4, 64, 2, 96), v_cache=z(4, 64, 2, 96))
    refused(UNSUPPORTED, k_cache=z(4, 32, 2, 128), v_cache=z(4, 32, 2, 128))
    ws, st = _space(c)
    for w, s in ((ws[:-1], st), (ws[1:], st)):
        assert m.idx_attn_paged_async(*c.args(), w, s, out_lse=c.lse, raise_on_error=False) == INVALID_ARGUMENT
    torch.cuda.synchronize()
    assert int(st.item()) == -7 and bool((c.out == 7).all())
    g = torch.cuda.CUDAGraph()
    s = torch.cuda.Stream()
    x = z(1)
    codes = []
    with torch.cuda.stream(s):
        with torch.cuda.graph(g, stream=s):
            x += 1
            codes.append(m.idx_attn_paged(*c.args(), raise_on_error=False))
    assert codes == [UNSUPPORTED]
    slots = z(1, 0, dt=torch.int32)
    assert m.idx_attn_selected(c.q, c.k, c.v, slots, 0.1, c.out, raise_on_error=False) == INVALID_ARGUMENT
    with pytest.raises(m.IdxError):
        m.idx_attn_selected(c.q, c.k, c.v, slots, 0.1, c.out)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("rows", [1, 2])
def test_paged_references_of_a_column(dtype, rows):
    """Scores that rise far above, or fall far below, those of the first positions, by tile and
    within one; a first key of -infinity; a first tile of nothing but -infinity."""
    import torch
    n = 900
    for kind in range(5):
        c = Case([n], [(0, 0, n)] * rows, 64, 1, 128, dtype)
        t = c.table.cpu()[0]
        pos = torch.arange(n)
        page, off = t[pos // PAGE].long().cuda(), (pos % PAGE).cuda()
        c.q.abs_()
        k = c.k[page, off].float() * 0.05
        ramp = torch.arange(n, device="cuda").float()[:, None, None]
        if kind == 0:
            k += ramp * 0.01                      # ever higher
        elif kind == 1:
            k += 9.0 - ramp * 0.01                # ever lower
        elif kind == 2:
            k[0] -= 20.0                          # the first far below the rest of its tile
        elif kind == 3:
            k[0] = -float("inf")
            k[500] += 12.0
        else:
            k[:130] = -float("inf")
        c.k[page, off] = k.to(_dt(dtype))
        assert run_paged(c) == 0
        if kind < 3:
            c.check()
        else:
            kk, vv = c.rows()[0]
            on = torch.isfinite(kk[:, 0, 0])
            for r in range(rows):
                want, wl, _, bo, bl, _ = A.attend(c.q[r], kk[on], vv[on], c.scale)
                assert bool(((c.out[r].double() - want).abs() <= bo).all()), (kind, r)
                assert bool(((c.lse[r].double() - wl).abs() <= bl).all()), (kind, r)
