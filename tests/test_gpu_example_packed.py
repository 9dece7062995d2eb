"""The decoding example's layer over a cache in 4 bits: what its last step wrote, and its attention against plain 64 bits."""
import importlib.util
import os

import pytest

from tests import append_ref as P, attn4_ref as A

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
PAGE = 64


def _example():
    spec = importlib.util.spec_from_file_location("decode_example", os.path.join(ROOT, "examples", "decode.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


@pytest.mark.parametrize("argv", [["--steps", "1"], ["--steps", "9", "--requests", "5", "--budget", "130"],
                                  ["--steps", "3", "--requests", "3", "--budget", "70", "--q-heads", "64", "--kv-heads", "1"]])
def test_packed_layer(argv):
    import torch
    ex = _example()
    args = ex.parse(argv + ["--packed"])
    packed = ex.packed_layer(args)
    first = packed.end.clone()
    ex.run(args, packed)
    assert int(packed.status.abs().max()) == 0
    assert torch.equal(packed.end, first + args.steps) and torch.equal(packed.pos, packed.end - 1)
    rows = []
    for t, n, v in zip(packed.table.long(), packed.end.tolist(), packed.v_in):
        pos = torch.arange(n, device="cuda")
        page, off = t[pos // PAGE], pos % PAGE
        rows.append((packed.k[page, off], packed.k_scale[page, off], packed.v[page, off], packed.v_scale[page, off]))
        # the last step's values lie in the last position
        codes, scales = P.quantise(v.double().cpu().numpy())
        at = rows[-1][2][-1].cpu().numpy(), rows[-1][3][-1].cpu().numpy()
        assert (P.values(P.unpack(at[0]), at[1]) == P.values(codes, scales)).all()
    A.check_rows(packed.q, packed.out, packed.lse, rows, packed.scale)


def test_main(capsys):
    _example().main(["--steps", "3", "--requests", "2", "--packed", "--time"])
    out = capsys.readouterr().out
    assert "4.25 bits an element" in out and "one step of the 3 layers" in out
