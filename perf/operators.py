"""The attention and cache operators on the sizes that they serve, in their plain form and through the library.

Three operators share one paged key-value cache [pages, 64 slots, key-value heads, head dimension]:

  paged     attention of one or a few new tokens over each request's cached window, the window split over the machine and
            joined; optionally the log-sum-exp of every head and the weight that every cached position received, added to
            a running total
  selected  attention of each row over its own list of physical slots (what the indexer's TopK returns, -1 = empty)
  evict     keeping a request's `budget` heaviest positions (its first and its most recent ones always), moved in order
            into fresh pages, with the new page table, lengths and weights

`own` false: elementary torch operations in 32 bits.  `own` true: the library's calls.
"""
import math

import torch

own = False

PAGE = 64
DTYPE = {"bf16": torch.bfloat16, "f16": torch.float16}


# ------------------------------------------------------------------ cases ----

def listed():
    return [
        # one token of one short conversation: latency is all that counts
        dict(name="paged-1x777-gqa", op="paged", requests=1, rows=1, lo=777, hi=777, window=0, edges=False, q_heads=32,
             kv_heads=8, dim=128, dtype="bf16", layout="slot", lse=True, weight=False),
        # the decode batch of the benchmark (32 requests x 2 rows, C4 lengths 4096..65536) with grouped heads
        dict(name="paged-32x2-gqa", op="paged", requests=32, rows=2, lo=4096, hi=65536, window=0, edges=False, q_heads=64,
             kv_heads=8, dim=128, dtype="bf16", layout="slot", lse=True, weight=False),
        # the same batch with the indexer's own head layout: 64 query heads on one key-value head
        dict(name="paged-32x2-mqa", op="paged", requests=32, rows=2, lo=4096, hi=65536, window=0, edges=False, q_heads=64,
             kv_heads=1, dim=128, dtype="bf16", layout="slot", lse=True, weight=False),
        # one very long context, one token: the split over the length carries it (an odd length, pages head by head)
        dict(name="paged-1x262143-f16", op="paged", requests=1, rows=1, lo=262143, hi=262143, window=0, edges=False,
             q_heads=64, kv_heads=8, dim=128, dtype="f16", layout="head", lse=True, weight=False),
        # many short ragged requests with a sliding window, a head of its own for every query head; requests of
        # length 0 and 1 among them; keys and values in one allocation
        dict(name="paged-48x3-mha-ragged", op="paged", requests=48, rows=3, lo=2, hi=3001, window=1000, edges=True,
             q_heads=16, kv_heads=16, dim=64, dtype="bf16", layout="joint", lse=True, weight=False),
        # a decode step that also adds up what every cached position received (the input of the eviction)
        dict(name="paged-16x1-weights", op="paged", requests=16, rows=1, lo=2048, hi=32768, window=0, edges=False,
             q_heads=32, kv_heads=8, dim=128, dtype="bf16", layout="slot", lse=True, weight=True),
        # one row over the slots that the indexer chose for it: the smallest sparse step
        dict(name="selected-1x512-mqa", op="selected", rows=1, topk=512, context=4096, q_heads=64, kv_heads=1, dim=128,
             dtype="bf16", layout="slot", short=False),
        # the decode batch's sparse step: 64 rows over 1024 slots of long contexts, some rows shorter than that
        dict(name="selected-64x1024-gqa", op="selected", rows=64, topk=1024, context=65536, q_heads=32, kv_heads=8, dim=128,
             dtype="f16", layout="head", short=True),
        # a prefill of 8192 rows over a context of 196,608 with 1024 slots a row (the benchmark's largest workload)
        dict(name="selected-8192x1024-mqa", op="selected", rows=8192, topk=1024, context=196608, q_heads=64, kv_heads=1,
             dim=128, dtype="bf16", layout="slot", short=False),
        # one conversation past its budget
        dict(name="evict-1x5001", op="evict", requests=1, lo=5001, hi=5001, budget=2000, first=4, last=64, kv_heads=8,
             dim=128, dtype="bf16", layout="slot"),
        # a whole batch cut down at once; a few requests are still within the budget and keep their pages
        dict(name="evict-32-to-8192", op="evict", requests=32, lo=4096, hi=65536, budget=8192, first=4, last=512,
             kv_heads=8, dim=128, dtype="bf16", layout="slot"),
        # a few very long contexts with one key-value head
        dict(name="evict-8x262144-mqa", op="evict", requests=8, lo=131072, hi=262144, budget=30001, first=1, last=1000,
             kv_heads=1, dim=128, dtype="f16", layout="head"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["paged", "paged", "selected", "evict"])
    dtype, layout = rng.choice(["bf16", "f16"]), rng.choice(["slot", "head", "joint"])
    dim = rng.choice([64, 128, 128, 256])
    kv_heads = rng.choice([1, 2, 4, 8])
    if op == "paged":
        q_heads = kv_heads * rng.choice([1, 2, 3, 4, 5, 8, 12, 16] + ([32, 64] if kv_heads == 1 else []))
        requests, hi = _log(rng, 1, 48), _log(rng, 1, 131072)
        while requests * hi * kv_heads * dim > 32 * 32768 * 8 * 128:
            requests, hi = max(1, requests // 2), max(1, hi * 3 // 4)
        weight = rng.random() < 0.3
        window = _log(rng, 1, 16384) if rng.random() < 0.3 else 0
        return dict(op=op, requests=requests, rows=rng.choice([1, 1, 2, 3, 4]), lo=rng.randint(0, hi), hi=hi,
                    window=window, edges=rng.random() < 0.3 and requests > 2, q_heads=q_heads, kv_heads=kv_heads, dim=dim,
                    dtype=dtype, layout=layout, lse=rng.random() < 0.7, weight=weight)
    if op == "selected":
        q_heads = kv_heads * rng.choice([1, 4, 7, 8, 16] + ([32, 64] if kv_heads == 1 else []))
        rows, topk = _log(rng, 1, 8192), rng.choice([512, 1024, _log(rng, 1, 2048)])
        context = max(topk, _log(rng, 512, 196608))
        while rows * topk * q_heads * dim > 8192 * 1024 * 64 * 128 // 2 or rows * topk * kv_heads * dim > 8192 * 1024 * 128:
            rows //= 2
        return dict(op=op, rows=max(1, rows), topk=topk, context=context, q_heads=q_heads, kv_heads=kv_heads, dim=dim,
                    dtype=dtype, layout=layout, short=rng.random() < 0.5)
    requests, hi = _log(rng, 1, 32), _log(rng, 64, 131072)
    while requests * hi * kv_heads * dim > 32 * 32768 * 8 * 128:
        requests, hi = max(1, requests // 2), max(64, hi * 3 // 4)
    budget = _log(rng, 16, max(17, hi // 2))
    first = rng.choice([0, 1, 4])
    return dict(op=op, requests=requests, lo=rng.randint(hi // 2, hi), hi=hi, budget=budget, first=first,
                last=rng.randint(0, budget - first), kv_heads=kv_heads, dim=dim, dtype=dtype, layout=layout)


def _lengths(c):
    """A request's cached positions: spread over lo..hi in no order; the first two 0 and 1 where the case has edges."""
    n, lo, hi = c["requests"], c["lo"], c["hi"]
    got = [lo + int((hi - lo) * ((0.5 + i * 0.6180339887498949) % 1.0)) for i in range(n)]
    if c.get("edges"):
        got[:2] = [0, 1]
    return got


def _windows(c):
    """(request, start, end) of each row: a request's last tokens, each sees what came before it."""
    got = []
    for i, n in enumerate(_lengths(c)):
        for j in range(c["rows"]):
            end = max(0, n - (c["rows"] - 1 - j))
            got.append((i, max(0, end - c["window"]) if c["window"] else 0, end))
    return got


def _row_slots(c):
    """How many slots each row of a selected case has: all, or for short rows what its place in the context leaves."""
    n, k = c["rows"], c["topk"]
    return [k if not c["short"] else min(k, int(k * 1.5 * ((0.5 + i * 0.6180339887498949) % 1.0))) for i in range(n)]


def work(c):
    d, h = c["dim"], c["kv_heads"]
    if c["op"] == "paged":
        rows, hq = _windows(c), c["q_heads"]
        seen = {}
        for i, a, b in rows:
            if b > a:
                p, q = seen.get(i, (a, b))
                seen[i] = (min(p, a), max(q, b))
        cached = sum(b - a for a, b in seen.values())
        pages = max(1, -(-max(_lengths(c)) // PAGE))
        bytes_ = cached * h * d * 2 * 2 + len(rows) * hq * d * 2 * 2 + sum(-(-b // PAGE) - a // PAGE for a, b in seen.values()) * 4
        bytes_ += len(rows) * (12 + hq * 4 * c["lse"])
        if c["weight"]:
            bytes_ += c["requests"] * pages * PAGE * 4 * 2
        return {"bytes": bytes_, "flops": sum(b - a for _, a, b in rows) * hq * d * 4}
    if c["op"] == "selected":
        n = sum(_row_slots(c))
        bytes_ = min(n, c["context"]) * h * d * 2 * 2 + c["rows"] * (c["topk"] * 4 + c["q_heads"] * (d * 2 * 2 + 4))
        return {"bytes": bytes_, "flops": n * c["q_heads"] * d * 4}
    lens = _lengths(c)
    cut = [n for n in lens if n > c["budget"]]
    pages = max(1, -(-max(lens) // PAGE))
    bytes_ = sum(lens) * 4 + len(lens) * pages * PAGE * 4 + len(lens) * (c["budget"] * 4 + pages * 8)
    return {"bytes": bytes_ + len(cut) * c["budget"] * h * d * 2 * 2 * 2, "flops": sum(cut)}


# ----------------------------------------------------------------- inputs ----

def _cache(pages, heads, dim, dtype, layout, g, fill=True):
    """Keys and values [pages, 64, heads, dim] as a program may hold them: slot by slot, head by head in a page, or both
    in one allocation."""
    make = (lambda *s: torch.randn(*s, device="cuda", dtype=dtype, generator=g)) if fill else \
        (lambda *s: torch.zeros(*s, device="cuda", dtype=dtype))
    if layout == "slot":
        return make(pages, PAGE, heads, dim), make(pages, PAGE, heads, dim)
    if layout == "head":
        return make(pages, heads, PAGE, dim).transpose(1, 2), make(pages, heads, PAGE, dim).transpose(1, 2)
    both = make(pages, 2, PAGE, heads, dim)
    return both[:, 0], both[:, 1]


def _page_table(lens, g, spare=0):
    """i32 [requests, pages of the longest]: every request's pages at random places, -1 behind them."""
    need = [-(-n // PAGE) for n in lens]
    total, width = max(1, sum(need)) + spare, max(1, max(need))
    perm = torch.randperm(total, device="cuda", generator=g).to(torch.int32)
    table = torch.full((len(lens), width), -1, dtype=torch.int32, device="cuda")
    at = 0
    for i, n in enumerate(need):
        table[i, :n] = perm[at:at + n]
        at += n
    return table, total


def _queries(rows, heads, dim, dtype, g):
    """Unit normal queries; the heads differ in how sharply they attend (a factor of 1/2 to 2)."""
    sharp = torch.exp2(torch.rand(heads, 1, device="cuda", generator=g) * 2 - 1)
    return (torch.randn(rows, heads, dim, device="cuda", generator=g) * sharp).to(dtype)


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    dtype, d, h = DTYPE[c["dtype"]], c["dim"], c["kv_heads"]
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    s = {"case": c, "scale": 1.0 / math.sqrt(d), "status": torch.zeros(1, dtype=torch.int32, device="cuda")}
    if c["op"] == "paged":
        lens, wins = _lengths(c), _windows(c)
        s["table"], pages = _page_table(lens, g)
        s["k"], s["v"] = _cache(pages, h, d, dtype, c["layout"], g)
        s["q"] = _queries(len(wins), c["q_heads"], d, dtype, g)
        s["req"], s["start"], s["end"] = i32([w[0] for w in wins]), i32([w[1] for w in wins]), i32([w[2] for w in wins])
        s["out"] = torch.empty_like(s["q"])
        s["lse"] = torch.empty(len(wins), c["q_heads"], device="cuda") if c["lse"] else None
        if c["weight"]:
            width = s["table"].shape[1] * PAGE
            s["win"] = torch.randn(len(lens), width, device="cuda", generator=g).mul_(2).exp_()
            s["wout"] = torch.empty_like(s["win"])
    elif c["op"] == "selected":
        table, pages = _page_table([c["context"]], g)
        s["k"], s["v"] = _cache(pages, h, d, dtype, c["layout"], g)
        s["q"] = _queries(c["rows"], c["q_heads"], d, dtype, g)
        # one position out of each of `topk` equal stretches of the context, in random order
        r, k, n = c["rows"], c["topk"], c["context"]
        edge = torch.arange(k + 1, device="cuda") * n // k
        pos = edge[:-1] + (torch.rand(r, k, device="cuda", generator=g) * (edge[1:] - edge[:-1])).long()
        pos = torch.minimum(pos, edge[1:] - 1)
        pos = pos.gather(1, torch.rand(r, k, device="cuda", generator=g).argsort(1))
        slots = table[0].long()[pos // PAGE] * PAGE + pos % PAGE
        have = i32(_row_slots(c))
        s["slots"] = torch.where(torch.arange(k, device="cuda")[None, :] < have[:, None], slots, -1).to(torch.int32)
        s["out"] = torch.empty_like(s["q"])
        s["lse"] = torch.empty(r, c["q_heads"], device="cuda")
    else:
        lens, n = _lengths(c), c["requests"]
        s["table"], pages = _page_table(lens, g)
        s["k"], s["v"] = _cache(pages, h, d, dtype, c["layout"], g)
        s["len"] = i32(lens)
        width = s["table"].shape[1] * PAGE
        # a few positions hold most of the weight; values of 8 significant bits, so that there are ties
        s["weight"] = torch.randn(n, width, device="cuda", generator=g).mul_(2).exp_().to(torch.bfloat16).float()
        per = -(-c["budget"] // PAGE)
        s["fresh"] = torch.randperm(n * per, device="cuda", generator=g).to(torch.int32).view(n, per)[:, : s["table"].shape[1]].contiguous()
        s["k_to"], s["v_to"] = _cache(n * per, h, d, dtype, c["layout"], g, fill=False)
        s["keep"] = torch.empty(n, c["budget"], dtype=torch.int32, device="cuda")
        s["new_len"] = torch.empty(n, dtype=torch.int32, device="cuda")
        s["new_table"] = torch.empty_like(s["table"])
        s["new_weight"] = torch.empty_like(s["weight"])
    return s


# -------------------------------------------------------------- operators ----

def _attend(q, k, v, valid, scale, dtype):
    """q [R, Hq, D], k and v [R, S, H, D], valid [R, S] -> out, log-sum-exp, weights [R, H, G, S]."""
    r, hq, d = q.shape
    h = k.shape[2]
    qf = q.float().view(r, h, hq // h, d)
    score = torch.matmul(qf, k.float().permute(0, 2, 3, 1)) * scale
    score = score.masked_fill(~valid[:, None, None, :], -math.inf)
    top = score.amax(-1, keepdim=True)
    top = torch.where(valid.any(1)[:, None, None, None], top, torch.zeros_like(top))
    p = torch.exp(score - top)
    total = p.sum(-1, keepdim=True)
    p = p / torch.where(valid.any(1)[:, None, None, None], total, torch.ones_like(total))
    vf = v.float().masked_fill(~valid[:, :, None, None], 0.0).transpose(1, 2)
    out = torch.matmul(p, vf).reshape(r, hq, d).to(dtype)
    lse = (top + torch.log(total)).reshape(r, hq)
    return out, lse, p


def _plain_paged(s):
    c, dev = s["case"], s["q"].device
    table, req = s["table"].long(), s["req"].long()
    pos = torch.arange(table.shape[1] * PAGE, device=dev)
    page, off = table[:, pos // PAGE].clamp(min=0)[req], (pos % PAGE)[None, :]
    valid = (pos[None, :] >= s["start"][:, None]) & (pos[None, :] < s["end"][:, None])
    out, lse, p = _attend(s["q"], s["k"][page, off], s["v"][page, off], valid, s["scale"], s["q"].dtype)
    got = {"out": out}
    if c["lse"]:
        got["lse"] = lse
    if c["weight"]:
        got["weight"] = s["win"] + torch.zeros_like(s["win"]).index_add_(0, req, p.sum((1, 2)))
    return got


def _plain_selected(s):
    slots = s["slots"].long()
    at = slots.clamp(min=0)
    out, lse, _ = _attend(s["q"], s["k"][at // PAGE, at % PAGE], s["v"][at // PAGE, at % PAGE], slots >= 0, s["scale"], s["q"].dtype)
    return {"out": out, "lse": lse}


def _plain_evict(s):
    c = s["case"]
    table, fresh, n = s["table"].long(), s["fresh"].long(), s["len"].long()[:, None]
    width, budget = s["weight"].shape[1], c["budget"]
    pos = torch.arange(width, device=table.device)[None, :]
    # heavier first, +0 above -0, NaN below every number; the kept ends above all, what is past the length below
    bits = s["weight"].view(torch.int32).long() & 0xFFFFFFFF
    key = torch.where(bits >= 1 << 31, 0xFFFFFFFF - bits, bits + (1 << 31))
    key = torch.where(s["weight"].isnan(), 0, key)
    key = torch.where((pos < c["first"]) | (pos >= n - c["last"]), 1 << 33, key)
    key = torch.where(pos < n, key, -1)
    best = torch.sort(key, dim=1, descending=True, stable=True).indices[:, :budget]
    best = torch.nn.functional.pad(best, (0, budget - best.shape[1]), value=width)
    keep = torch.sort(torch.where(best < n, best, width), dim=1).values
    new_len = torch.clamp(n, max=budget)
    rank = torch.arange(budget, device=table.device)[None, :]
    keep = torch.where(rank < new_len, keep, -1)
    at, cut = keep.clamp(min=0), (n > budget) & (rank < new_len)
    page, to = torch.gather(table, 1, at // PAGE), fresh[:, (torch.arange(budget, device=table.device) // PAGE).clamp(max=fresh.shape[1] - 1)]
    to_off = (rank % PAGE).expand_as(to)
    s["k_to"][to[cut], to_off[cut]] = s["k"][page[cut], (at % PAGE)[cut]]
    s["v_to"][to[cut], to_off[cut]] = s["v"][page[cut], (at % PAGE)[cut]]
    moved = torch.nn.functional.pad(fresh, (0, table.shape[1] - fresh.shape[1]), value=-1)
    weight = torch.where(rank < new_len, torch.gather(s["weight"], 1, at), 0.0)[:, :width]
    return {"keep": keep.to(torch.int32), "len": new_len[:, 0].to(torch.int32),
            "table": torch.where(n > budget, moved, table).to(torch.int32),
            "weight": torch.nn.functional.pad(weight, (0, width - weight.shape[1])), "k": s["k_to"], "v": s["v_to"]}


def _own_paged(s):
    import fp4_sparse_attention_tma_gb300 as m
    c, q = s["case"], s["q"]
    if "work" not in s:
        s["work"] = torch.empty(m.idx_attn_paged_scratch_bytes(q.shape[0], q.shape[1], c["kv_heads"], q.shape[2], *s["table"].shape,
                                                               with_weights=c["weight"]), dtype=torch.uint8, device=q.device)
    m.idx_attn_paged_async(q, s["k"], s["v"], s["table"], s["req"], s["start"], s["end"], s["scale"], s["out"], s["work"], s["status"],
                           out_lse=s["lse"], weight_in=s.get("win"), weight_out=s.get("wout"))
    got = {"out": s["out"]}
    if c["lse"]:
        got["lse"] = s["lse"]
    if c["weight"]:
        got["weight"] = s["wout"]
    return got


def _own_selected(s):
    import fp4_sparse_attention_tma_gb300 as m
    c, q = s["case"], s["q"]
    if "work" not in s:
        s["work"] = torch.empty(m.idx_attn_selected_scratch_bytes(q.shape[0], q.shape[1], c["kv_heads"], q.shape[2], c["topk"]),
                                dtype=torch.uint8, device=q.device)
    m.idx_attn_selected_async(q, s["k"], s["v"], s["slots"], s["scale"], s["out"], s["work"], s["status"], out_lse=s["lse"])
    return {"out": s["out"], "lse": s["lse"]}


def _own_evict(s):
    import fp4_sparse_attention_tma_gb300 as m
    c = s["case"]
    if "work" not in s:
        s["work"] = torch.empty(m.idx_cache_evict_scratch_bytes(*s["table"].shape, s["k_to"].shape[0], c["budget"]),
                                dtype=torch.uint8, device=s["k"].device)
    m.idx_cache_evict_async(s["k"], s["v"], s["table"], s["len"], s["weight"], c["budget"], c["first"], c["last"], s["k_to"], s["v_to"],
                            s["fresh"], s["keep"], s["new_len"], s["new_table"], s["new_weight"], s["work"], s["status"])
    return {"keep": s["keep"], "len": s["new_len"], "table": s["new_table"], "weight": s["new_weight"], "k": s["k_to"], "v": s["v_to"]}


def run(state):
    op = state["case"]["op"]
    if own:
        return {"paged": _own_paged, "selected": _own_selected, "evict": _own_evict}[op](state)
    return {"paged": _plain_paged, "selected": _plain_selected, "evict": _plain_evict}[op](state)


# ------------------------------------------------------------- in 64 bits ----

def _exact_rows(q, k, v, scale):
    """q [R, Hq, D], k and v [R, S, H, D] in 64 bits: softmax(q k^T scale) v, log-sum-exp and weights [R, Hq, S]."""
    groups = q.shape[1] // k.shape[2]
    kk, vv = k.repeat_interleave(groups, 2).permute(0, 2, 1, 3), v.repeat_interleave(groups, 2).permute(0, 2, 1, 3)
    score = (kk @ q[..., None])[..., 0] * scale if k.shape[2] > 1 else q @ k[:, :, 0].transpose(1, 2) * scale
    lse = torch.logsumexp(score, -1)
    p = torch.exp(score - lse[..., None])
    out = (p[:, :, None] @ vv)[:, :, 0] if k.shape[2] > 1 else p @ v[:, :, 0]
    return out, lse, p


def exact(case, seed):
    c, s = case, prepare(case, seed)
    f8 = lambda t: t.to(torch.float64)  # noqa: E731
    if c["op"] == "paged":
        q = f8(s["q"])
        out, lse = torch.zeros_like(q), torch.full(q.shape[:2], -math.inf, dtype=torch.float64, device="cuda")
        total = f8(s["win"]) if c["weight"] else None
        for r, (i, a, b) in enumerate(_windows(c)):
            if b <= a:
                continue
            pos = torch.arange(a, b, device="cuda")
            page = s["table"][i].long()[pos // PAGE]
            o, m, p = _exact_rows(q[r:r + 1], f8(s["k"][page, pos % PAGE])[None], f8(s["v"][page, pos % PAGE])[None], s["scale"])
            out[r], lse[r] = o[0], m[0]
            if total is not None:
                total[i, a:b] += p[0].sum(0)
        got = {"out": out}
        if c["lse"]:
            got["lse"] = lse
        if c["weight"]:
            got["weight"] = total
        return got
    if c["op"] == "selected":
        q = f8(s["q"])
        out, lse = torch.zeros_like(q), torch.full(q.shape[:2], -math.inf, dtype=torch.float64, device="cuda")
        have = _row_slots(c)
        r = 0
        while r < c["rows"]:  # rows with equally many slots go together
            e, n = r + 1, have[r]
            while e < c["rows"] and e - r < 256 and have[e] == n:
                e += 1
            if n:
                at = s["slots"][r:e, :n].long()
                out[r:e], lse[r:e], _ = _exact_rows(q[r:e], f8(s["k"][at // PAGE, at % PAGE]), f8(s["v"][at // PAGE, at % PAGE]), s["scale"])
            r = e
        return {"out": out, "lse": lse}
    k_to, v_to, weight = f8(s["k_to"]), f8(s["v_to"]), torch.zeros_like(s["new_weight"], dtype=torch.float64)
    for i, n in enumerate(_lengths(c)):
        w = f8(s["weight"][i, :n])
        if n <= c["budget"]:
            weight[i, :n] = w
            continue
        ends = torch.arange(n, device="cuda")
        ends = (ends < c["first"]) | (ends >= n - c["last"])
        order = torch.sort(torch.where(ends, math.inf, w), descending=True, stable=True).indices[: c["budget"]]
        kept = torch.sort(order).values
        weight[i, : c["budget"]] = w[kept]
        to = torch.arange(c["budget"], device="cuda")
        page, fresh = s["table"][i].long()[kept // PAGE], s["fresh"][i].long()[to // PAGE]
        k_to[fresh, to % PAGE] = f8(s["k"][page, kept % PAGE])
        v_to[fresh, to % PAGE] = f8(s["v"][page, kept % PAGE])
    return {"keep": None, "len": None, "table": None, "weight": weight, "k": k_to, "v": v_to}
