"""Writing a paged cache and attending over one held in 4 bits, on the sizes that they serve, in their plain form and through
the library.

The cache is paged [pages, 64 slots, key-value heads, head dimension], in 16 bits, or in 4: E2M1 codes [.., D / 2] (the even
element in the low half of a byte) with one UE8M0 scale byte for 32 elements [.., D / 32], the format of the indexer's keys.

  append     new tokens' queries and keys normed head by head and rotated by their positions, keys and values written to
             their requests' pages
  append4    the same into a 4-bit cache; the appended slots are then read back
  gather4    listed slots of a 4-bit cache as 16-bit rows
  paged4     attention of one or a few new tokens over each request's window of a 4-bit cache
  selected4  attention of each row over its own list of physical slots of a 4-bit cache (-1 = empty)

`own` false: elementary torch operations in 32 bits (the sums of squares in 64: a key in 4 bits may lie next to a border).
`own` true: the library's calls.
"""
import math

import torch

own = False

PAGE = 64
BLOCK = 32
DTYPE = {"bf16": torch.bfloat16, "f16": torch.float16}
EPS = 1e-6


# ------------------------------------------------------------------ cases ----

def listed():
    return [
        # one new token for each of four conversations, queries included: latency is all that counts
        dict(name="append-4x1", op="append", requests=4, rows=1, lo=500, hi=4000, edges=False, q_heads=32, kv_heads=8, dim=128,
             dtype="bf16", layout="slot", norm=True, rot=128, first=0, pairs=False),
        # a prompt's chunk of 8192 tokens in four requests, 64 query heads on 8
        dict(name="append-4x2048", op="append", requests=4, rows=2048, lo=0, hi=2047, edges=False, q_heads=64, kv_heads=8, dim=128,
             dtype="bf16", layout="slot", norm=True, rot=128, first=0, pairs=False),
        # a decode batch of 32 requests x 2 tokens into a 4-bit cache; the last 64 dimensions rotated in neighbouring pairs
        dict(name="append4-32x2", op="append4", requests=32, rows=2, lo=100, hi=4096, edges=False, q_heads=64, kv_heads=8, dim=128,
             dtype="bf16", layout="slot", norm=True, rot=64, first=64, pairs=True),
        # ragged prompts of 48 requests x 171 tokens, fp16, a key-value head for two query heads, keys and values of a page together
        dict(name="append4-48x171", op="append4", requests=48, rows=171, lo=0, hi=777, edges=True, q_heads=16, kv_heads=8, dim=64,
             dtype="f16", layout="joint", norm=False, rot=64, first=0, pairs=False),
        # what the indexer chose for one row
        dict(name="gather4-512", op="gather4", slots=512, context=4096, kv_heads=1, dim=128, dtype="bf16", layout="slot", holes=False),
        # a long request's cache read back in whole, in the order of its pages' slots; some entries empty
        dict(name="gather4-65536", op="gather4", slots=65535, context=65536, kv_heads=8, dim=128, dtype="bf16", layout="head", holes=True),
        # one token of one short conversation
        dict(name="paged4-1x777-gqa", op="paged4", requests=1, rows=1, lo=777, hi=777, window=0, edges=False, q_heads=32, kv_heads=8,
             dim=128, dtype="bf16", layout="slot"),
        # the decode batch of the benchmark (32 requests x 2 rows, C4 lengths 4096..65536) with grouped heads
        dict(name="paged4-32x2-gqa", op="paged4", requests=32, rows=2, lo=4096, hi=65536, window=0, edges=False, q_heads=64, kv_heads=8,
             dim=128, dtype="bf16", layout="slot"),
        # the same batch with the indexer's own head layout, fp16: 64 query heads on one key-value head
        dict(name="paged4-32x2-mqa", op="paged4", requests=32, rows=2, lo=4096, hi=65536, window=0, edges=False, q_heads=64, kv_heads=1,
             dim=128, dtype="f16", layout="slot"),
        # many short ragged requests with a sliding window, a head of its own for every query head; lengths 0 and 1 among them
        dict(name="paged4-48x3-mha-ragged", op="paged4", requests=48, rows=3, lo=2, hi=3001, window=1000, edges=True, q_heads=16,
             kv_heads=16, dim=64, dtype="bf16", layout="joint"),
        # the decode batch's sparse step: 64 rows over 1024 slots of long contexts, some rows shorter than that
        dict(name="selected4-64x1024-gqa", op="selected4", rows=64, topk=1024, context=65536, q_heads=32, kv_heads=8, dim=128,
             dtype="f16", layout="head", short=True),
        # a prefill of 8192 rows over a context of 196,608 with 1024 slots a row (the benchmark's largest workload)
        dict(name="selected4-8192x1024-mqa", op="selected4", rows=8192, topk=1024, context=196608, q_heads=64, kv_heads=1, dim=128,
             dtype="bf16", layout="slot", short=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "append4", "gather4", "paged4", "paged4", "selected4"])
    dtype, layout = rng.choice(["bf16", "f16"]), rng.choice(["slot", "head", "joint"])
    dim = rng.choice([64, 128, 128, 256])
    kv_heads = rng.choice([1, 2, 4, 8])
    if op in ("append", "append4"):
        q_heads = kv_heads * rng.choice([1, 2, 3, 4, 7, 8])
        requests, rows = _log(rng, 1, 64), _log(rng, 1, 4096)
        while requests * rows * (q_heads + 2 * kv_heads) * dim > 4 * 2048 * 80 * 128:
            rows = max(1, rows // 2)
        rot = rng.choice([0, 32, 64, dim])
        hi = _log(rng, 1, 4096)
        return dict(op=op, requests=requests, rows=rows, lo=rng.randint(0, hi), hi=hi, edges=rng.random() < 0.3 and requests > 2,
                    q_heads=q_heads, kv_heads=kv_heads, dim=dim, dtype=dtype, layout=layout, norm=rot == 0 or rng.random() < 0.7, rot=rot,
                    first=rng.choice([0, dim - rot]), pairs=rng.random() < 0.5)
    if op == "gather4":
        slots, context = _log(rng, 1, 65536), _log(rng, 512, 65536)
        return dict(op=op, slots=slots, context=context, kv_heads=kv_heads, dim=min(dim, 128), dtype=dtype, layout=layout,
                    holes=rng.random() < 0.5)
    if op == "paged4":
        q_heads = kv_heads * rng.choice([1, 2, 3, 4, 5, 8, 12, 16] + ([32, 64] if kv_heads == 1 else []))
        requests, hi = _log(rng, 1, 48), _log(rng, 1, 131072)
        while requests * hi * kv_heads * dim > 32 * 32768 * 8 * 128:
            requests, hi = max(1, requests // 2), max(1, hi * 3 // 4)
        window = _log(rng, 1, 16384) if rng.random() < 0.3 else 0
        return dict(op=op, requests=requests, rows=rng.choice([1, 1, 2, 3, 4]), lo=rng.randint(0, hi), hi=hi, window=window,
                    edges=rng.random() < 0.3 and requests > 2, q_heads=q_heads, kv_heads=kv_heads, dim=dim, dtype=dtype, layout=layout)
    q_heads = kv_heads * rng.choice([1, 4, 7, 8, 16] + ([32, 64] if kv_heads == 1 else []))
    rows, topk = _log(rng, 1, 8192), rng.choice([512, 1024, _log(rng, 1, 2048)])
    context = max(topk, _log(rng, 512, 196608))
    while rows * topk * q_heads * dim > 8192 * 1024 * 64 * 128 // 2 or rows * topk * kv_heads * dim > 8192 * 1024 * 128:
        rows //= 2
    return dict(op=op, rows=max(1, rows), topk=topk, context=context, q_heads=q_heads, kv_heads=kv_heads, dim=dim, dtype=dtype,
                layout=layout, short=rng.random() < 0.5)


def _spread(n, lo, hi):
    return [lo + int((hi - lo) * ((0.5 + i * 0.6180339887498949) % 1.0)) for i in range(n)]


def _lengths(c):
    """A request's cached positions: spread over lo..hi in no order; the first two 0 and 1 where the case has edges."""
    got = _spread(c["requests"], c["lo"], c["hi"])
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
    packed = d // 2 + d // BLOCK   # bytes of a head's 4-bit row
    if c["op"] in ("append", "append4"):
        rows, hq = c["requests"] * c["rows"], c["q_heads"]
        bytes_ = rows * (hq * d * 2 * 2 + h * d * 2 * 2 + 8) + min(rows, max(_lengths(c)) + c["rows"]) * c["rot"] * 4
        bytes_ += rows * h * 2 * (d * 2 if c["op"] == "append" else packed * 2 + d * 2)
        return {"bytes": bytes_, "flops": rows * (hq + h) * d * (3 * c["norm"] + 3 * (c["rot"] > 0))}
    if c["op"] == "gather4":
        return {"bytes": c["slots"] * (4 + h * 2 * d * 2) + min(c["slots"], c["context"]) * h * 2 * packed, "flops": c["slots"] * h * 2 * d}
    if c["op"] == "paged4":
        rows, hq = _windows(c), c["q_heads"]
        seen = {}
        for i, a, b in rows:
            if b > a:
                p, q = seen.get(i, (a, b))
                seen[i] = (min(p, a), max(q, b))
        cached = sum(b - a for a, b in seen.values())
        bytes_ = cached * h * packed * 2 + len(rows) * hq * d * 2 * 2 + sum(-(-b // PAGE) - a // PAGE for a, b in seen.values()) * 4
        return {"bytes": bytes_ + len(rows) * (12 + hq * 4), "flops": sum(b - a for _, a, b in rows) * hq * d * 4}
    n = sum(_row_slots(c))
    bytes_ = min(n, c["context"]) * h * packed * 2 + c["rows"] * (c["topk"] * 4 + c["q_heads"] * (d * 2 * 2 + 4))
    return {"bytes": bytes_, "flops": n * c["q_heads"] * d * 4}


# ---------------------------------------------------------- the 4-bit form ----

def _quantise(x):
    """x [.., D] float32 -> codes u8 [.., D / 2], scales u8 [.., D / 32]: 2^e with the smallest e >= -127 such that no element
    exceeds 6 2^e, elements to the nearest of 0, 0.5, 1, 1.5, 2, 3, 4, 6, ties to the even code."""
    b = x.reshape(*x.shape[:-1], -1, BLOCK)
    part, exp = torch.frexp(b.abs().amax(-1, keepdim=True))       # part in [0.5, 1); 6 = 0.75 * 2^3
    e = torch.where(part == 0, -127, torch.clamp(exp - 3 + (part > 0.75).int(), min=-127))
    y = torch.ldexp(b, -e)
    a = y.abs()
    code = torch.zeros_like(a, dtype=torch.uint8)
    for at in (0.25, 1.25, 2.5, 5.0):                            # here the tie's even code is the lower one
        code += a > at
    for at in (0.75, 1.75, 3.5):                                 # and here the upper
        code += a >= at
    code = (code + 8 * (y < 0).to(torch.uint8)).reshape(*x.shape[:-1], -1, 2)
    return code[..., 0] + 16 * code[..., 1], (e[..., 0] + 127).to(torch.uint8)


def _table(dtype, device):
    """The two values of each byte of codes [256, 2]."""
    v = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], dtype=dtype, device=device)
    v = torch.cat([v, -v])
    at = torch.arange(256, device=device)
    return torch.stack([v[at % 16], v[at // 16]], 1)


def _values(codes, scales, dtype=torch.float32):
    """The numbers that codes [.., D / 2] and scales [.., D / 32] stand for, [.., D]."""
    x = _table(dtype, codes.device)[codes.int()].reshape(*scales.shape, BLOCK)
    return x.mul_(torch.pow(torch.tensor(2.0, dtype=dtype, device=codes.device), scales.to(dtype) - 127)[..., None]).flatten(-2)


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


def _cache4(pages, heads, dim, layout, g, fill=True):
    """The same in 4 bits: (codes, scales) of keys and of values; normal values, a few channels larger than the others."""
    dev = "cuda"
    shape = (pages, heads, PAGE) if layout == "head" else (pages, PAGE, heads)
    parts = []
    both_c = torch.zeros(pages, 2, *shape[1:], dim // 2, dtype=torch.uint8, device=dev) if layout == "joint" else None
    both_s = torch.zeros(pages, 2, *shape[1:], dim // BLOCK, dtype=torch.uint8, device=dev) if layout == "joint" else None
    for i in range(2):
        codes = both_c[:, i] if both_c is not None else torch.zeros(*shape, dim // 2, dtype=torch.uint8, device=dev)
        scales = both_s[:, i] if both_s is not None else torch.zeros(*shape, dim // BLOCK, dtype=torch.uint8, device=dev)
        if fill:
            loud = torch.exp2(2 * torch.randn(dim, device=dev, generator=g).clamp(min=0))
            step = max(1, (1 << 26) // (PAGE * heads * dim))
            for a in range(0, pages, step):
                b = min(pages, a + step)
                codes[a:b], scales[a:b] = _quantise(torch.randn(b - a, *shape[1:], dim, device=dev, generator=g) * (loud if i == 0 else 1.0))
        parts.append((codes.transpose(1, 2), scales.transpose(1, 2)) if layout == "head" else (codes, scales))
    return parts


def _page_table(lens, g):
    """i32 [requests, pages of the longest]: every request's pages at random places, -1 behind them."""
    need = [-(-n // PAGE) for n in lens]
    total, width = max(1, sum(need)), max(1, max(need))
    perm = torch.randperm(total, device="cuda", generator=g).to(torch.int32)
    table = torch.full((len(lens), width), -1, dtype=torch.int32, device="cuda")
    at = 0
    for i, n in enumerate(need):
        table[i, :n] = perm[at:at + n]
        at += n
    return table, total


def _queries(rows, heads, dim, dtype, g, loud=1.0):
    """Unit normal queries; the heads differ in how sharply they attend (a factor of 1/2 to 2)."""
    sharp = torch.exp2(torch.rand(heads, 1, device="cuda", generator=g) * 2 - 1) * loud
    return (torch.randn(rows, heads, dim, device="cuda", generator=g) * sharp).to(dtype)


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    dtype, d, h = DTYPE[c["dtype"]], c["dim"], c["kv_heads"]
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    s = {"case": c, "scale": 1.0 / math.sqrt(d), "status": torch.zeros(1, dtype=torch.int32, device="cuda")}
    if c["op"] in ("append", "append4"):
        old, n = _lengths(c), c["rows"]
        s["table"], pages = _page_table([x + n for x in old], g)
        wide = torch.randn(c["requests"] * n, c["q_heads"] + 2 * h, d, device="cuda", generator=g).to(dtype)   # a fused projection
        s["q"], s["k"], s["v"] = wide.split([c["q_heads"], h, h], 1)
        s["req"] = i32([i for i in range(c["requests"]) for _ in range(n)])
        s["pos"] = i32([x + j for x in old for j in range(n)])
        if c["norm"]:
            s["q_weight"], s["k_weight"] = (1 + 0.2 * torch.randn(2, d, device="cuda", generator=g)).to(dtype)
        if c["rot"]:
            angle = torch.arange(max(old) + n, device="cuda", dtype=torch.float64)[:, None] * \
                10000.0 ** (-torch.arange(c["rot"] // 2, device="cuda", dtype=torch.float64) / (c["rot"] // 2))
            s["rope"] = torch.stack([angle.cos(), angle.sin()], 1).float()
        s["out_q"] = torch.empty(c["requests"] * n, c["q_heads"], d, device="cuda", dtype=dtype)
        if c["op"] == "append":
            s["kc"], s["vc"] = _cache(pages, h, d, dtype, c["layout"], g)
        else:
            (s["kc"], s["ks"]), (s["vc"], s["vs"]) = _cache4(pages, h, d, c["layout"], g, fill=False)
            s["slots"] = s["table"][s["req"].long(), s["pos"].long() // PAGE] * PAGE + s["pos"] % PAGE
            s["out_k"], s["out_v"] = torch.empty(2, c["requests"] * n, h, d, device="cuda", dtype=dtype)
        return s
    if c["op"] == "gather4":
        table, pages = _page_table([c["context"]], g)
        (s["kc"], s["ks"]), (s["vc"], s["vs"]) = _cache4(pages, h, d, c["layout"], g)
        pos = torch.arange(c["slots"], device="cuda") * c["context"] // c["slots"]
        slots = table[0][pos // PAGE] * PAGE + (pos % PAGE).to(torch.int32)
        if c["holes"]:
            slots[torch.rand(c["slots"], device="cuda", generator=g) < 0.05] = -1
        s["slots"] = slots
        s["out_k"], s["out_v"] = torch.empty(2, c["slots"], h, d, device="cuda", dtype=dtype)
        return s
    if c["op"] == "paged4":
        lens, wins = _lengths(c), _windows(c)
        s["table"], pages = _page_table(lens, g)
        rows = len(wins)
        s["req"], s["start"], s["end"] = i32([w[0] for w in wins]), i32([w[1] for w in wins]), i32([w[2] for w in wins])
    else:
        table, pages = _page_table([c["context"]], g)
        rows = c["rows"]
        # one position out of each of `topk` equal stretches of the context, in random order
        r, k, n = rows, c["topk"], c["context"]
        edge = torch.arange(k + 1, device="cuda") * n // k
        pos = edge[:-1] + (torch.rand(r, k, device="cuda", generator=g) * (edge[1:] - edge[:-1])).long()
        pos = torch.minimum(pos, edge[1:] - 1)
        pos = pos.gather(1, torch.rand(r, k, device="cuda", generator=g).argsort(1))
        slots = table[0].long()[pos // PAGE] * PAGE + pos % PAGE
        have = i32(_row_slots(c))
        s["slots"] = torch.where(torch.arange(k, device="cuda")[None, :] < have[:, None], slots, -1).to(torch.int32)
    (s["kc"], s["ks"]), (s["vc"], s["vs"]) = _cache4(pages, h, d, c["layout"], g)
    s["q"] = _queries(rows, c["q_heads"], d, dtype, g, 0.4)
    s["out"] = torch.empty_like(s["q"])
    s["lse"] = torch.empty(rows, c["q_heads"], device="cuda")
    return s


# -------------------------------------------------------------- operators ----

def _normed(x, weight):
    """x / sqrt(mean x^2 + eps) * weight over the last dimension, in 32 bits from a sum in 64."""
    x = x.float()
    if weight is None:
        return x
    mean = x.double().square().sum(-1, keepdim=True).float() / x.shape[-1]
    return x * (1.0 / torch.sqrt(mean + EPS)) * weight.float()


def _rotated(x, rope, first, pairs):
    """x [R, H, D] with the dimensions first .. first + rot turned by the rows' angles, rope [R, 2, rot / 2]."""
    if rope is None:
        return x
    half = rope.shape[2]
    cos, sin = rope[:, None, 0], rope[:, None, 1]
    x = x.clone()
    y = x[..., first:first + 2 * half]
    a, b = (y[..., 0::2].clone(), y[..., 1::2].clone()) if pairs else (y[..., :half].clone(), y[..., half:].clone())
    low, high = a * cos - b * sin, b * cos + a * sin
    if pairs:
        y[..., 0::2], y[..., 1::2] = low, high
    else:
        y[..., :half], y[..., half:] = low, high
    return x


def _plain_append(s):
    c = s["case"]
    pos = s["pos"].long()
    rope = s["rope"][pos] if c["rot"] else None
    make = lambda x, w: _rotated(_normed(x, s.get(w)), rope, c["first"], c["pairs"])  # noqa: E731
    q, k = make(s["q"], "q_weight").to(s["q"].dtype), make(s["k"], "k_weight")
    page, off = s["table"].long()[s["req"].long(), pos // PAGE], pos % PAGE
    if c["op"] == "append":
        s["kc"][page, off] = k.to(s["q"].dtype)
        s["vc"][page, off] = s["v"]
        return {"q": q, "k": s["kc"], "v": s["vc"]}
    s["kc"][page, off], s["ks"][page, off] = _quantise(k)
    s["vc"][page, off], s["vs"][page, off] = _quantise(s["v"].float())
    back = lambda x, y: _values(x[page, off], y[page, off]).to(s["q"].dtype)  # noqa: E731
    return {"q": q, "k": back(s["kc"], s["ks"]), "v": back(s["vc"], s["vs"])}


def _plain_gather4(s):
    slots = s["slots"].long()
    at, there = slots.clamp(min=0), (slots >= 0)[:, None, None]
    back = lambda x, y: torch.where(there, _values(x[at // PAGE, at % PAGE], y[at // PAGE, at % PAGE]), 0.0).to(s["out_k"].dtype)  # noqa: E731
    return {"k": back(s["kc"], s["ks"]), "v": back(s["vc"], s["vs"])}


def _attend(q, k, v, valid, scale, dtype):
    """q [R, Hq, D], k and v [R, S, H, D], valid [R, S] -> out, log-sum-exp."""
    r, hq, d = q.shape
    h = k.shape[2]
    qf = q.float().view(r, h, hq // h, d)
    score = torch.matmul(qf, k.permute(0, 2, 3, 1)) * scale
    score = score.masked_fill(~valid[:, None, None, :], -math.inf)
    top = score.amax(-1, keepdim=True)
    top = torch.where(valid.any(1)[:, None, None, None], top, torch.zeros_like(top))
    p = torch.exp(score - top)
    total = p.sum(-1, keepdim=True)
    p = p / torch.where(valid.any(1)[:, None, None, None], total, torch.ones_like(total))
    out = torch.matmul(p, v.transpose(1, 2)).reshape(r, hq, d).to(dtype)
    return out, (top + torch.log(total)).reshape(r, hq)


def _plain_paged4(s):
    dev = s["q"].device
    table, req = s["table"].long(), s["req"].long()
    pos = torch.arange(table.shape[1] * PAGE, device=dev)
    page, off = table[:, pos // PAGE].clamp(min=0)[req], (pos % PAGE)[None, :]
    valid = (pos[None, :] >= s["start"][:, None]) & (pos[None, :] < s["end"][:, None])
    out, lse = _attend(s["q"], _values(s["kc"], s["ks"])[page, off], _values(s["vc"], s["vs"])[page, off], valid, s["scale"], s["q"].dtype)
    return {"out": out, "lse": lse}


def _plain_selected4(s):
    slots = s["slots"].long()
    at = slots.clamp(min=0)
    out, lse = _attend(s["q"], _values(s["kc"], s["ks"])[at // PAGE, at % PAGE], _values(s["vc"], s["vs"])[at // PAGE, at % PAGE],
                       slots >= 0, s["scale"], s["q"].dtype)
    return {"out": out, "lse": lse}


def _own_append(s):
    import fp4_sparse_attention_tma_gb300 as m
    c = s["case"]
    more = dict(q=s["q"], out_q=s["out_q"], q_weight=s.get("q_weight"), k_weight=s.get("k_weight"), eps=EPS, rope=s.get("rope"),
                rope_first=c["first"], rope_pairs=c["pairs"])
    if c["op"] == "append":
        m.idx_cache_append_async(s["k"], s["v"], s["table"], s["req"], s["pos"], s["kc"], s["vc"], s["status"], **more)
        return {"q": s["out_q"], "k": s["kc"], "v": s["vc"]}
    m.idx_cache_append_fp4_async(s["k"], s["v"], s["table"], s["req"], s["pos"], s["kc"], s["ks"], s["vc"], s["vs"], s["status"], **more)
    m.idx_cache_gather_fp4_async(s["kc"], s["ks"], s["vc"], s["vs"], s["slots"], s["out_k"], s["out_v"], s["status"])
    return {"q": s["out_q"], "k": s["out_k"], "v": s["out_v"]}


def _own_gather4(s):
    import fp4_sparse_attention_tma_gb300 as m
    m.idx_cache_gather_fp4_async(s["kc"], s["ks"], s["vc"], s["vs"], s["slots"], s["out_k"], s["out_v"], s["status"])
    return {"k": s["out_k"], "v": s["out_v"]}


def _own_paged4(s):
    import fp4_sparse_attention_tma_gb300 as m
    c, q = s["case"], s["q"]
    if "work" not in s:
        s["work"] = torch.empty(m.idx_attn_paged_fp4_scratch_bytes(q.shape[0], q.shape[1], c["kv_heads"], q.shape[2], *s["table"].shape),
                                dtype=torch.uint8, device=q.device)
    m.idx_attn_paged_fp4_async(q, s["kc"], s["ks"], s["vc"], s["vs"], s["table"], s["req"], s["start"], s["end"], s["scale"], s["out"],
                               s["work"], s["status"], out_lse=s["lse"])
    return {"out": s["out"], "lse": s["lse"]}


def _own_selected4(s):
    import fp4_sparse_attention_tma_gb300 as m
    c, q = s["case"], s["q"]
    if "work" not in s:
        s["work"] = torch.empty(m.idx_attn_selected_fp4_scratch_bytes(q.shape[0], q.shape[1], c["kv_heads"], q.shape[2], c["topk"]),
                                dtype=torch.uint8, device=q.device)
    m.idx_attn_selected_fp4_async(q, s["kc"], s["ks"], s["vc"], s["vs"], s["slots"], s["scale"], s["out"], s["work"], s["status"],
                                  out_lse=s["lse"])
    return {"out": s["out"], "lse": s["lse"]}


def run(state):
    op = state["case"]["op"]
    if own:
        return {"append": _own_append, "append4": _own_append, "gather4": _own_gather4, "paged4": _own_paged4,
                "selected4": _own_selected4}[op](state)
    return {"append": _plain_append, "append4": _plain_append, "gather4": _plain_gather4, "paged4": _plain_paged4,
            "selected4": _plain_selected4}[op](state)


# ------------------------------------------------------------- in 64 bits ----

def _exact_rows(q, k, v, scale):
    """q [R, Hq, D], k and v [R, S, H, D] in 64 bits: softmax(q k^T scale) v and the log-sum-exp."""
    groups = q.shape[1] // k.shape[2]
    kk, vv = k.repeat_interleave(groups, 2).permute(0, 2, 1, 3), v.repeat_interleave(groups, 2).permute(0, 2, 1, 3)
    score = (kk @ q[..., None])[..., 0] * scale if k.shape[2] > 1 else q @ k[:, :, 0].transpose(1, 2) * scale
    lse = torch.logsumexp(score, -1)
    p = torch.exp(score - lse[..., None])
    return (p[:, :, None] @ vv)[:, :, 0] if k.shape[2] > 1 else p @ v[:, :, 0], lse


def _exact_nearest(x):
    """x [.., D] in 64 bits -> the numbers that its 4-bit form stands for."""
    b = x.unflatten(-1, (-1, BLOCK))
    top = b.abs().amax(-1, keepdim=True)
    e = torch.ceil(torch.log2(top / 6))
    e = torch.where(top > 6 * torch.exp2(e), e + 1, torch.where(top <= 6 * torch.exp2(e - 1), e - 1, e))   # where the logarithm rounds
    unit = torch.where(top > 0, torch.exp2(e.clamp(min=-127)), 1.0)
    a = (b / unit).abs()
    step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0))
    return (torch.copysign(torch.round(a / step) * step, b) * unit).flatten(-2)   # (round: ties to the even multiple)


def _exact_turned(x, weight, c, s):
    x = x.double()
    if weight is not None:
        x = x * (x * x).mean(-1, keepdim=True).add(EPS).rsqrt() * weight.double()
    n, first = c["rot"] // 2, c["first"]
    if n:
        turn = torch.complex(*(t.double() for t in s["rope"][s["pos"].long()].unbind(1)))[:, None]
        at = torch.arange(n, device=x.device)
        i, j = (first + 2 * at, first + 2 * at + 1) if c["pairs"] else (first + at, first + n + at)
        z = torch.complex(x[..., i], x[..., j]) * turn
        x = x.clone()
        x[..., i], x[..., j] = z.real, z.imag
    return x


def exact(case, seed):
    c, s = case, prepare(case, seed)
    f8 = lambda t: t.to(torch.float64)  # noqa: E731
    if c["op"] in ("append", "append4"):
        q, k = _exact_turned(s["q"], s.get("q_weight"), c, s), _exact_turned(s["k"], s.get("k_weight"), c, s)
        if c["op"] == "append4":
            return {"q": q, "k": _exact_nearest(k), "v": _exact_nearest(f8(s["v"]))}
        kc, vc = f8(s["kc"]), f8(s["vc"])
        for i in range(c["requests"]):
            mine = s["req"] == i
            pos = s["pos"][mine].long()
            page = s["table"][i].long()[pos // PAGE]
            kc[page, pos % PAGE], vc[page, pos % PAGE] = k[mine], f8(s["v"][mine])
        return {"q": q, "k": kc, "v": vc}
    if c["op"] == "gather4":
        at = s["slots"].long()
        got = {}
        for name, codes, scales in (("k", s["kc"], s["ks"]), ("v", s["vc"], s["vs"])):
            x = torch.zeros(c["slots"], c["kv_heads"], c["dim"], dtype=torch.float64, device="cuda")
            on = at >= 0
            x[on] = _values(codes[at[on] // PAGE, at[on] % PAGE], scales[at[on] // PAGE, at[on] % PAGE], torch.float64)
            got[name] = x
        return got
    q = f8(s["q"])
    out, lse = torch.zeros_like(q), torch.full(q.shape[:2], -math.inf, dtype=torch.float64, device="cuda")
    wide = lambda codes, scales, page, off: _values(codes[page, off], scales[page, off], torch.float64)  # noqa: E731
    if c["op"] == "paged4":
        for r, (i, a, b) in enumerate(_windows(c)):
            if b <= a:
                continue
            pos = torch.arange(a, b, device="cuda")
            page = s["table"][i].long()[pos // PAGE]
            o, m = _exact_rows(q[r:r + 1], wide(s["kc"], s["ks"], page, pos % PAGE)[None], wide(s["vc"], s["vs"], page, pos % PAGE)[None],
                               s["scale"])
            out[r], lse[r] = o[0], m[0]
        return {"out": out, "lse": lse}
    have, r = _row_slots(c), 0
    while r < c["rows"]:  # rows with equally many slots go together
        e, n = r + 1, have[r]
        while e < c["rows"] and e - r < 256 and have[e] == n:
            e += 1
        if n:
            at = s["slots"][r:e, :n].long()
            out[r:e], lse[r:e] = _exact_rows(q[r:e], wide(s["kc"], s["ks"], at // PAGE, at % PAGE), wide(s["vc"], s["vs"], at // PAGE, at % PAGE),
                                             s["scale"])
        r = e
    return {"out": out, "lse": lse}
