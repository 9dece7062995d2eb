"""The decoding example: its last step against plain 64-bit attention, the pages it holds, and
the weights that a request's kept positions carry on."""
import importlib.util
import os

import pytest

from tests import attn_ref as A

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
PAGE = 64


def _example():
    spec = importlib.util.spec_from_file_location("decode_example", os.path.join(ROOT, "examples", "decode.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


@pytest.mark.parametrize("argv", [["--steps", "3"], ["--steps", "41", "--slack", "9", "--requests", "5", "--budget", "130"]])
def test_decode_example(argv):
    import torch
    ex = _example()
    args = ex.parse(argv)
    sparse, dense = ex.run(args)
    rows = []
    for s in sparse.slots.long():
        s = s[s >= 0]
        rows.append((sparse.k[s // PAGE, s % PAGE], sparse.v[s // PAGE, s % PAGE]))
    assert all(k.shape[0] == args.topk for k, _ in rows)
    A.check_rows(sparse.q, sparse.out, sparse.lse, rows, sparse.scale)
    rows = []
    for t, n in zip(dense.host_table, dense.lengths):
        pos = torch.arange(n)
        page = torch.tensor(t)[pos // PAGE].cuda()
        rows.append((dense.k[page, (pos % PAGE).cuda()], dense.v[page, (pos % PAGE).cuda()]))
    A.check_rows(dense.q, dense.out, dense.lse, rows, dense.scale)
    # no page twice, and none lost
    held = [x for t in dense.host_table for x in t]
    assert len(set(held + dense.free)) == len(held) + len(dense.free) == dense.pages
    assert dense.evictions == (0 if args.steps == 3 else 4)
    # every step adds a weight of 1 a query head and request; an eviction only drops some
    total, most = dense.weight.double().sum(1), args.steps * args.q_heads
    assert bool((total <= most * (1 + 1e-4)).all())
    if dense.evictions == 0:
        assert bool((total >= most * (1 - 1e-4)).all())
    else:
        assert bool((total >= 0.25 * most).all())
    tail = torch.arange(dense.weight.shape[1], device="cuda")[None] >= torch.tensor(dense.lengths, device="cuda")[:, None]
    assert bool((dense.weight[tail] == 0).all())
