"""Eviction from the paged cache by accumulated weight against a plain selection: lengths,
budgets, ties, signed zeros and NaN, layouts, fresh pages in the same or another pool, long
contexts, graphs, and what the call refuses."""
import numpy as np
import pytest

from tests import attn_ref as A
from tests.test_gpu_attention import PAGE, make_cache

pytestmark = pytest.mark.gpu

INVALID_ARGUMENT, UNSUPPORTED, INVALID_METADATA, INVALID_PAGE = 1, 2, 3, 4


class Case:
    def __init__(self, lens, budget, first=0, last=0, hk=2, dim=64, dtype=None, layout="slot", pool="other", seed=1, spare=0,
                 kind="mixed"):
        import torch
        dtype = dtype or torch.bfloat16
        rng = np.random.default_rng(seed)
        need = [-(-n // PAGE) for n in lens]
        self.mp = max(1, max(need)) + spare
        self.dp = min(self.mp, -(-budget // PAGE) + spare)
        cut = [n > budget for n in lens]
        src = max(1, sum(need))
        fresh = len(lens) * self.dp
        total = src + (fresh if pool == "same" else 0)
        perm = rng.permutation(total)
        self.h_table = np.full((len(lens), self.mp), -1, dtype=np.int32)
        at = 0
        for i, n in enumerate(need):
            self.h_table[i, :n] = perm[at:at + n]
            at += n
        self.k, self.v = make_cache(total, hk, dim, dtype, layout, seed)
        if pool == "same":
            self.k_to, self.v_to = self.k, self.v
            free = perm[src:]
        else:
            self.k_to, self.v_to = make_cache(fresh, hk, dim, dtype, layout, seed + 7)
            free = rng.permutation(fresh)
        self.h_fresh = free.astype(np.int32).reshape(len(lens), self.dp)
        w = np.exp(2 * rng.standard_normal((len(lens), self.mp * PAGE))).astype(np.float32)
        if kind == "mixed":    # ties, zeros of both signs, NaN, infinities
            w = np.round(w * 4) / 4
            pick = rng.integers(0, 40, w.shape)
            for code, x in ((0, 0.0), (1, -0.0), (2, np.nan), (3, np.inf), (4, -1.0), (5, -np.inf)):
                w = np.where(pick == code, np.float32(x), w)
        elif kind == "equal":
            w[:] = 1.0
        self.h_weight = w.astype(np.float32)
        i32 = lambda x: torch.from_numpy(np.ascontiguousarray(np.asarray(x, dtype=np.int32))).cuda()
        self.table, self.fresh, self.len = i32(self.h_table), i32(self.h_fresh), i32(lens)
        self.weight = torch.from_numpy(self.h_weight).cuda()
        self.lens, self.budget, self.first, self.last = lens, budget, first, last
        n = len(lens)
        self.keep = torch.full((n, budget), 7, dtype=torch.int32, device="cuda")
        self.new_len = torch.full((n,), 7, dtype=torch.int32, device="cuda")
        self.new_table = torch.full((n, self.mp), 7, dtype=torch.int32, device="cuda")
        self.new_weight = torch.full((n, self.mp * PAGE), 7.0, device="cuda")
        self.before = (self.k.clone(), self.v.clone())
        self.to_before = (self.k_to.clone(), self.v_to.clone())

    def args(self):
        return (self.k, self.v, self.table, self.len, self.weight, self.budget, self.first, self.last, self.k_to, self.v_to,
                self.fresh, self.keep, self.new_len, self.new_table, self.new_weight)

    def run(self):
        import torch
        import fp4_sparse_attention_tma_gb300 as m
        code = m.idx_cache_evict(*self.args(), raise_on_error=False)
        torch.cuda.synchronize()
        return code

    def check(self):
        import torch
        keep, weight = self.keep.cpu().numpy(), self.new_weight.cpu().numpy()
        want_k, want_v = (t.clone() for t in self.to_before)
        for i, n in enumerate(self.lens):
            kept = A.keep_positions(self.h_weight[i], n, self.budget, self.first, self.last)
            m = len(kept)
            assert keep[i, :m].tolist() == kept, i
            assert (keep[i, m:] == -1).all()
            assert int(self.new_len[i]) == m
            want_w = np.zeros(self.mp * PAGE, dtype=np.float32)
            want_w[:m] = self.h_weight[i][kept]
            assert np.array_equal(weight[i].view(np.uint32), want_w.view(np.uint32)), i
            table = self.new_table[i].cpu().numpy()
            if n <= self.budget:
                assert np.array_equal(table, self.h_table[i])
                continue
            assert np.array_equal(table[:self.dp], self.h_fresh[i]) and (table[self.dp:] == -1).all()
            kept = torch.tensor(kept)
            to = torch.arange(m)
            sp = torch.from_numpy(self.h_table[i])[kept // PAGE].long().cuda()
            dp = torch.from_numpy(self.h_fresh[i])[to // PAGE].long().cuda()
            for want, src in ((want_k, self.before[0]), (want_v, self.before[1])):
                want[dp, (to % PAGE).cuda()] = src[sp, (kept % PAGE).cuda()]
        # every byte of the destination pool: what was not written is as it was
        assert torch.equal(self.k_to.view(torch.int16), want_k.view(torch.int16))
        assert torch.equal(self.v_to.view(torch.int16), want_v.view(torch.int16))


@pytest.mark.parametrize("pool", ["other", "same"])
@pytest.mark.parametrize("layout", ["slot", "head", "joint"])
@pytest.mark.parametrize("budget,first,last", [(1, 0, 0), (1, 1, 0), (37, 4, 8), (64, 0, 0), (65, 0, 65), (128, 64, 64),
                                               (200, 1, 150)])
def test_evict(pool, layout, budget, first, last):
    lens = [0, 1, 36, 37, 38, 64, 65, 129, 200, 201, 1000]
    c = Case(lens, budget, first, last, layout=layout, pool=pool, spare=1)
    assert c.run() == 0
    c.check()


@pytest.mark.parametrize("kind", ["mixed", "equal", "smooth"])
@pytest.mark.parametrize("heads,dim", [(1, 256), (3, 128), (8, 64)])
def test_evict_weights_and_heads(kind, heads, dim):
    import torch
    c = Case([5000, 17000, 4096, 4097], 2049, 4, 64, hk=heads, dim=dim, dtype=torch.float16, kind=kind)
    assert c.run() == 0
    c.check()


@pytest.mark.parametrize("n,budget", [(70001, 1000), (70001, 69999), (401000, 30001)])
def test_evict_long(n, budget):
    """Contexts spread over a cluster, the last beyond what its shared memory holds."""
    c = Case([n, n // 3], budget, 1, 100, hk=1)
    assert c.run() == 0
    c.check()


def test_evict_budget_above_everything():
    c = Case([100, 30], 1000, 2, 2)
    assert c.dp * PAGE < 1000
    assert c.run() == 0
    c.check()


def test_evict_then_attend():
    """The table, lengths and pages that come out serve the next attention call."""
    import torch
    import fp4_sparse_attention_tma_gb300 as m
    c = Case([900, 50], 130, 2, 30, hk=2, dim=128, pool="same", kind="smooth")
    assert c.run() == 0
    q = torch.randn(2, 8, 128, device="cuda").to(torch.bfloat16)
    out = torch.empty_like(q)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
    m.idx_attn_paged(q, c.k, c.v, c.new_table, i32([0, 1]), i32([0, 0]), c.new_len, 0.09, out)
    rows = []
    for i, n in enumerate(c.lens):
        kept = torch.tensor(A.keep_positions(c.h_weight[i], n, 130, 2, 30))
        pg = torch.from_numpy(c.h_table[i])[kept // PAGE].long().cuda()
        rows.append((c.before[0][pg, (kept % PAGE).cuda()], c.before[1][pg, (kept % PAGE).cuda()]))
    A.check_rows(q, out, None, rows, 0.09)


def test_evict_stream_ordered_and_graph():
    import torch
    import fp4_sparse_attention_tma_gb300 as m
    c = Case([3000, 100, 700], 257, 4, 16)
    ws = torch.full((m.idx_cache_evict_scratch_bytes(3, c.mp, c.k_to.shape[0], 257),), 0xA5, dtype=torch.uint8, device="cuda")
    st = torch.full((1,), -7, dtype=torch.int32, device="cuda")
    assert m.idx_cache_evict_async(*c.args(), ws, st) == 0
    torch.cuda.synchronize()
    assert int(st.item()) == 0
    c.check()
    s, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.stream(s):
        with torch.cuda.graph(g, stream=s):
            assert m.idx_cache_evict_async(*c.args(), ws, st) == 0
    for t in (c.keep, c.new_len, c.new_table):
        t.fill_(7)
    st.fill_(-7)
    g.replay()
    torch.cuda.synchronize()
    assert int(st.item()) == 0
    c.check()


def test_evict_device_errors_move_nothing():
    def failed(code, change, pool="other"):
        import torch
        c = Case([300, 100, 500], 130, pool=pool)
        change(c)
        assert c.run() == code
        assert bool((c.keep == -1).all()) and bool((c.new_len == -1).all()) and bool((c.new_table == -1).all())
        assert bool(c.new_weight.isnan().all())
        assert torch.equal(c.k_to.view(torch.int16), c.to_before[0].view(torch.int16))
        assert torch.equal(c.v_to.view(torch.int16), c.to_before[1].view(torch.int16))

    def put(t, i, x):
        t[i] = x

    failed(INVALID_METADATA, lambda c: put(c.len, 1, -1))
    failed(INVALID_METADATA, lambda c: put(c.len, 1, c.mp * PAGE + 1))
    failed(INVALID_PAGE, lambda c: put(c.table, (0, 4), -1))
    failed(INVALID_PAGE, lambda c: put(c.table, (1, 1), c.k.shape[0]))
    failed(INVALID_PAGE, lambda c: put(c.fresh, (0, 2), c.k_to.shape[0]))
    failed(INVALID_PAGE, lambda c: put(c.fresh, (0, 2), -1))
    failed(INVALID_PAGE, lambda c: put(c.fresh, (0, 2), c.fresh[0, 0]))       # named twice
    failed(INVALID_PAGE, lambda c: put(c.fresh, (0, 2), c.fresh[2, 0]))       # by two requests
    failed(INVALID_PAGE, lambda c: put(c.fresh, (0, 2), c.table[1, 0]), pool="same")   # another request's page
    c = Case([300, 100, 500], 130)
    c.fresh[1, :] = -5                  # a request that is not cut: never read
    c.h_fresh[1, :] = -5
    assert c.run() == 0
    c.check()


def test_evict_refused_arguments():
    import torch
    import fp4_sparse_attention_tma_gb300 as m
    c = Case([300, 100], 130)
    names = ["k_cache", "v_cache", "page_table", "seq_len", "weight", "budget", "keep_first", "keep_last", "k_dst", "v_dst",
             "dst_page_table", "out_keep_idx", "out_len", "out_page_table", "out_weight"]

    def refused(code=INVALID_ARGUMENT, **kw):
        got = m.idx_cache_evict(**{**dict(zip(names, c.args())), **kw}, raise_on_error=False)
        torch.cuda.synchronize()
        assert got == code, (kw.keys(), got)
        assert bool((c.keep == 7).all()) and bool((c.new_len == 7).all())

    refused(budget=0)
    refused(keep_first=-1)
    refused(keep_first=100, keep_last=31)
    refused(budget=129)                                  # not the width of out_keep_idx
    refused(weight=c.weight[:, :-1].contiguous())
    refused(weight=c.weight.double())
    refused(dst_page_table=c.fresh[:, :2].contiguous())  # too few fresh pages
    refused(k_dst=c.k)                                   # one of the two caches only
    refused(k_dst=c.v_to)                                # keys and values to one place
    refused(k_dst=c.k[1:], v_dst=c.v[1:])                # neither the caches nor apart from them
    refused(out_page_table=c.table)
    refused(out_weight=c.weight)
    refused(v_cache=c.v.half())
    refused(k_dst=c.k_to[:, :1].expand(-1, PAGE, -1, -1))


def test_evict_many_requests():
    """More requests than a wave of clusters, short and long."""
    rng = np.random.default_rng(8)
    lens = [int(x) for x in rng.integers(0, 400, 700)]
    c = Case(lens, 100, 2, 10, hk=1, pool="same")
    assert c.run() == 0
    c.check()


def test_evict_large_pool():
    """A pool whose bitmap of fresh pages does not fit shared memory."""
    import torch
    import fp4_sparse_attention_tma_gb300 as m
    c = Case([500, 100, 300], 130, hk=1)
    pages = 1_700_000
    kd = torch.zeros(pages, PAGE, 1, 64, dtype=torch.bfloat16, device="cuda")
    vd = torch.zeros_like(kd)
    far = torch.arange(c.fresh.numel(), device="cuda", dtype=torch.int32).view_as(c.fresh) * 7 + (pages - 7 * c.fresh.numel())
    args = list(c.args())
    args[8], args[9], args[10] = kd, vd, far
    assert m.idx_cache_evict(*args) == 0
    torch.cuda.synchronize()
    for i in (0, 2):
        kept = torch.tensor(A.keep_positions(c.h_weight[i], c.lens[i], 130, 0, 0))
        sp = torch.from_numpy(c.h_table[i])[kept // PAGE].long().cuda()
        to = torch.arange(130, device="cuda")
        got = kd[far[i][to // PAGE].long(), to % PAGE]
        assert torch.equal(got.view(torch.int16), c.k[sp, (kept % PAGE).cuda()].view(torch.int16))
    args[10] = far.clone()
    args[10][0, 1] = far[2, 0]           # named by two requests
    assert m.idx_cache_evict(*args, raise_on_error=False) == INVALID_PAGE
