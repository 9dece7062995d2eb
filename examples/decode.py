"""Decoding with a bounded cache: attention layers on the library's operators.

  sparse layer   the FP4 indexer picks each row's slots (idx_topk_fp4_prefill_async), and
                 idx_attn_selected_async attends over exactly those: the slots are physical,
                 so they index the layer's key-value pages as they are
  dense layer    idx_attn_paged_async attends over everything that a request has cached and
                 adds up what every position received; when a request has grown past
                 budget + slack, idx_cache_evict_async keeps its `budget` positions of
                 largest weight (its first and most recent ones always) in fresh pages;
                 idx_cache_append_async norms new queries and keys and writes new tokens
  packed layer   (--packed) a cache in 4 bits: idx_cache_append_fp4_async norms and rotates a
                 prompt's or a step's queries and keys and writes codes and scales, and
                 idx_attn_paged_fp4_async attends over them

The layers of a step are stream-ordered and synchronise nothing; the step is captured into
a CUDA graph once and replayed, with lengths, page table and new tokens written into the
same buffers between replays.  Inputs are synthetic.

    python examples/decode.py --requests 4 --context 2000 --steps 40
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import fp4_sparse_attention_tma_gb300 as m  # noqa: E402
from fp4_sparse_attention_tma_gb300 import inputs  # noqa: E402

PAGE = 64


class SparseLayer:
    """The indexer's selection, then attention over it: 64 query heads on one key-value head."""

    def __init__(self, requests, context, topk, seed):
        p = inputs.make_problem(seed, [context] * requests, [[(0, context)]] * requests, topk)
        dev = lambda a: torch.from_numpy(a).cuda()
        self.index = dict(q_fp4=dev(p.q_fp4), q_scale=dev(p.q_scale), k_cache_fp4=dev(p.k_cache_fp4), k_scale=dev(p.k_scale),
                          weights=dev(p.weights), page_table=dev(p.page_table), row_req=dev(p.row_req),
                          row_start=dev(p.row_start), row_end=dev(p.row_end))
        R, D = p.rows, 128
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        rand = lambda *s: torch.randn(*s, device="cuda", generator=g).to(torch.bfloat16)
        self.k, self.v, self.q = rand(p.num_pages, PAGE, 1, D), rand(p.num_pages, PAGE, 1, D), rand(R, 64, D)
        self.scale, self.topk = D ** -0.5, topk
        self.slots = torch.empty(R, topk, dtype=torch.int32, device="cuda")
        self.out, self.lse = torch.empty_like(self.q), torch.empty(R, 64, device="cuda")
        space = lambda n: torch.empty(n, dtype=torch.uint8, device="cuda")
        self.pick_space = space(m.idx_topk_fp4_scratch_bytes(R, topk))
        self.attn_space = space(m.idx_attn_selected_scratch_bytes(R, 64, 1, D, topk))
        self.status = torch.zeros(2, 1, dtype=torch.int32, device="cuda")

    def step(self):
        m.idx_topk_fp4_prefill_async(**self.index, topk=self.topk, out_phys_slot=self.slots, workspace=self.pick_space,
                                     status=self.status[0])
        m.idx_attn_selected_async(self.q, self.k, self.v, self.slots, self.scale, self.out, self.attn_space, self.status[1],
                                  out_lse=self.lse)


class DenseLayer:
    """A paged cache that grows by a token a step and is cut to `budget` where it has grown past its limit."""

    def __init__(self, lengths, q_heads, kv_heads, dim, budget, slack, first, last, seed):
        R = len(lengths)
        self.budget, self.limit, self.first, self.last = budget, budget + slack, first, last
        self.mp = -(-(max(max(lengths), self.limit) + 1) // PAGE)
        per = -(-budget // PAGE)
        self.pages = R * (self.mp + per)
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        self.rand = lambda *s: torch.randn(*s, device="cuda", generator=g).to(torch.bfloat16)
        both = self.rand(self.pages, 2, PAGE, kv_heads, dim)          # keys and values of a page in one piece
        self.k, self.v = both[:, 0], both[:, 1]
        self.free = list(range(self.pages))
        self.lengths = list(lengths)
        self.host_table = [[self.free.pop() for _ in range(-(-n // PAGE))] for n in lengths]
        i32 = lambda *s: torch.zeros(*s, dtype=torch.int32, device="cuda")
        self.table, self.fresh = i32(R, self.mp), i32(R, per)
        self.req, self.start, self.end = torch.arange(R, dtype=torch.int32, device="cuda"), i32(R), i32(R)
        self.weight = torch.zeros(R, self.mp * PAGE, device="cuda")
        self.new_weight = torch.zeros_like(self.weight)
        self.keep, self.new_len, self.new_table = i32(R, budget), i32(R), i32(R, self.mp)
        self.q = self.rand(R, q_heads, dim)
        self.q_weight, self.k_weight = 1 + 0.1 * self.rand(dim), 1 + 0.1 * self.rand(dim)
        self.out, self.lse = torch.empty_like(self.q), torch.empty(R, q_heads, device="cuda")
        self.scale = dim ** -0.5
        space = lambda n: torch.empty(n, dtype=torch.uint8, device="cuda")
        self.attn_space = space(m.idx_attn_paged_scratch_bytes(R, q_heads, kv_heads, dim, R, self.mp, with_weights=True))
        self.evict_space = space(m.idx_cache_evict_scratch_bytes(R, self.mp, self.pages, budget))
        self.status = torch.zeros(3, 1, dtype=torch.int32, device="cuda")
        self.evictions = 0
        self._upload()

    def _upload(self):
        rows = [t + [-1] * (self.mp - len(t)) for t in self.host_table]
        self.table.copy_(torch.tensor(rows, dtype=torch.int32))
        self.end.copy_(torch.tensor(self.lengths, dtype=torch.int32))

    def append(self):
        """A new token's key, value and query for every request."""
        R = len(self.lengths)
        for i in range(R):
            if self.lengths[i] % PAGE == 0:
                self.host_table[i].append(self.free.pop())
        pos = torch.tensor(self.lengths, dtype=torch.int32, device="cuda")
        self.lengths = [n + 1 for n in self.lengths]
        self._upload()
        new = self.rand(R, *self.k.shape[2:])
        m.idx_cache_append_async(new, self.rand(*new.shape), self.table, self.req, pos, self.k, self.v, self.status[2],
                                 q=self.rand(*self.q.shape), out_q=self.q, q_weight=self.q_weight, k_weight=self.k_weight,
                                 eps=1e-6)

    def step(self):
        m.idx_attn_paged_async(self.q, self.k, self.v, self.table, self.req, self.start, self.end, self.scale, self.out,
                               self.attn_space, self.status[0], out_lse=self.lse, weight_in=self.weight,
                               weight_out=self.weight)

    def evict(self):
        """Cuts every request that is longer than the budget, once one has reached the limit."""
        if max(self.lengths) < self.limit:
            return False
        cut = [n > self.budget for n in self.lengths]
        taken = [[self.free.pop() for _ in range(self.fresh.shape[1])] if c else [-1] * self.fresh.shape[1] for c in cut]
        self.fresh.copy_(torch.tensor(taken, dtype=torch.int32))
        m.idx_cache_evict_async(self.k, self.v, self.table, self.end, self.weight, self.budget, self.first, self.last, self.k,
                                self.v, self.fresh, self.keep, self.new_len, self.new_table, self.new_weight,
                                self.evict_space, self.status[1])
        self.weight.copy_(self.new_weight)
        if int(self.status[1].item()) != 0:
            raise RuntimeError(m.idx_topk_status_string(int(self.status[1].item())))
        for i, c in enumerate(cut):
            if c:
                self.free += self.host_table[i]
                self.host_table[i], self.lengths[i] = taken[i], self.budget
        self._upload()
        self.evictions += 1
        return True


class PackedLayer:
    """A paged cache in 4 bits that starts with a prompt of every request and grows by a token a step."""

    def __init__(self, lengths, steps, q_heads, kv_heads, dim, seed):
        R = len(lengths)
        self.mp = -(-(max(lengths) + steps) // PAGE)
        pages = R * self.mp
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        self.rand = lambda *s: torch.randn(*s, device="cuda", generator=g).to(torch.bfloat16)
        u8 = lambda *s: torch.zeros(*s, dtype=torch.uint8, device="cuda")
        i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
        self.k, self.v = u8(pages, PAGE, kv_heads, dim // 2), u8(pages, PAGE, kv_heads, dim // 2)
        self.k_scale, self.v_scale = u8(pages, PAGE, kv_heads, dim // 32), u8(pages, PAGE, kv_heads, dim // 32)
        self.table = torch.randperm(pages, device="cuda", generator=g).to(torch.int32).view(R, self.mp)
        self.weights = dict(q_weight=1 + 0.1 * self.rand(dim), k_weight=1 + 0.1 * self.rand(dim), eps=1e-6)
        angles = torch.arange(self.mp * PAGE, device="cuda")[:, None] * 10000.0 ** (-torch.arange(dim // 2, device="cuda") * 2 / dim)
        self.rope = torch.stack([angles.cos(), angles.sin()], 1).float()
        self.scale = dim ** -0.5
        # the step's own buffers
        self.q_in, self.k_in, self.v_in = self.rand(R, q_heads, dim), self.rand(R, kv_heads, dim), self.rand(R, kv_heads, dim)
        self.q, self.out = torch.empty_like(self.q_in), torch.empty_like(self.q_in)
        self.lse = torch.empty(R, q_heads, device="cuda")
        self.req, self.start = torch.arange(R, dtype=torch.int32, device="cuda"), i32([0] * R)
        self.pos, self.end = i32([n - 1 for n in lengths]), i32(lengths)
        self.attn_space = torch.empty(m.idx_attn_paged_fp4_scratch_bytes(R, q_heads, kv_heads, dim, R, self.mp),
                                      dtype=torch.uint8, device="cuda")
        self.status = torch.zeros(2, 1, dtype=torch.int32, device="cuda")
        # the prompts, in one call: every request's keys and values, whatever its length
        rows = [(r, n) for r, length in enumerate(lengths) for n in range(length)]
        req, pos = i32([r for r, _ in rows]), i32([n for _, n in rows])
        m.idx_cache_append_fp4(self.rand(len(rows), kv_heads, dim), self.rand(len(rows), kv_heads, dim), self.table, req, pos,
                               self.k, self.k_scale, self.v, self.v_scale, k_weight=self.weights["k_weight"],
                               eps=self.weights["eps"], rope=self.rope)

    def append(self):
        """A new token's query, key and value for every request, into the step's buffers."""
        for x in (self.q_in, self.k_in, self.v_in):
            x.copy_(self.rand(*x.shape))
        self.pos += 1
        self.end += 1

    def step(self):
        m.idx_cache_append_fp4_async(self.k_in, self.v_in, self.table, self.req, self.pos, self.k, self.k_scale, self.v,
                                     self.v_scale, self.status[0], q=self.q_in, out_q=self.q, rope=self.rope, **self.weights)
        m.idx_attn_paged_fp4_async(self.q, self.k, self.k_scale, self.v, self.v_scale, self.table, self.req, self.start,
                                   self.end, self.scale, self.out, self.attn_space, self.status[1], out_lse=self.lse)


def packed_layer(args):
    lengths = [max(1, args.budget - 7 * i) for i in range(args.requests)]
    return PackedLayer(lengths, args.steps, args.q_heads, args.kv_heads, 128, seed=args.seed + 2)


def run(args, packed=None):
    """Runs the steps, a packed layer's with them; returns the two other layers as the last step left them."""
    sparse = SparseLayer(args.requests, args.context, args.topk, args.seed)
    lengths = [max(1, args.budget - 7 * i) for i in range(args.requests)]
    dense = DenseLayer(lengths, args.q_heads, args.kv_heads, 128, args.budget, args.slack, first=4, last=args.budget // 8,
                       seed=args.seed + 1)
    layers = [sparse, dense] + ([packed] if packed else [])
    graph, side = None, torch.cuda.Stream()
    for n in range(args.steps):
        dense.append()
        if packed:
            packed.append()
        if graph is None:
            # two steps run as they are (and set the kernels up); then the step is captured, which runs nothing
            for layer in layers:
                layer.step()
            if n == 1:
                torch.cuda.synchronize()
                graph = torch.cuda.CUDAGraph()
                with torch.cuda.stream(side), torch.cuda.graph(graph, stream=side):
                    for layer in layers:
                        layer.step()
                torch.cuda.synchronize()
        else:
            graph.replay()
        bad = torch.cat([sparse.status, dense.status[:1], dense.status[2:]] + ([packed.status] if packed else [])).max()
        if n + 1 < args.steps:
            dense.evict()
        if int(bad.item()) != 0:
            raise RuntimeError(m.idx_topk_status_string(int(bad.item())))
    torch.cuda.synchronize()
    if graph is not None and args.time:
        t0, t1 = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        t0.record()
        for _ in range(20):
            graph.replay()
        t1.record()
        torch.cuda.synchronize()
        print("one step of the %d layers: %.1f us (replays back to back)" % (len(layers), t0.elapsed_time(t1) / 20 * 1e3))
    return sparse, dense


def parse(argv=None):
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--requests", type=int, default=4)
    ap.add_argument("--context", type=int, default=4096, help="positions of the sparse layer's requests")
    ap.add_argument("--topk", type=int, default=512, choices=[512, 1024])
    ap.add_argument("--budget", type=int, default=512, help="positions that the dense layer keeps of a request")
    ap.add_argument("--slack", type=int, default=16, help="how far a request grows past the budget before it is cut")
    ap.add_argument("--steps", type=int, default=40)
    ap.add_argument("--q-heads", type=int, default=32)
    ap.add_argument("--kv-heads", type=int, default=8)
    ap.add_argument("--seed", type=int, default=1)
    ap.add_argument("--packed", action="store_true", help="a layer over a cache in 4 bits beside the two")
    ap.add_argument("--time", action="store_true", help="time the captured step afterwards (its weights go on adding up)")
    return ap.parse_args(argv)


def main(argv=None):
    args = parse(argv)
    packed = packed_layer(args) if args.packed else None
    sparse, dense = run(args, packed)
    print("%d steps, %d evictions, lengths %s, %d pages free" % (args.steps, dense.evictions, dense.lengths, len(dense.free)))
    print("sparse layer: |out| %.4f; dense layer: |out| %.4f, weight added up %.1f" % (
        float(sparse.out.float().abs().mean()), float(dense.out.float().abs().mean()), float(dense.weight.sum())))
    if packed:
        print("packed layer: |out| %.4f, %.2f bits an element" % (
            float(packed.out.float().abs().mean()), 8 * (packed.k.nbytes + packed.k_scale.nbytes) / (2 * packed.k.numel())))


if __name__ == "__main__":
    main()
