"""What the cache-writing calls refuse, found by their argument checks before any device work (CPU: descriptors of host
tensors; a call that passes the checks ends with the code of the missing device instead)."""
import pytest
import torch

import fp4_sparse_attention_tma_gb300 as m

INVALID, UNSUPPORTED, OVERFLOW = 1, 2, 5
PASSED = (6, 1)   # no device (CUDA error); with one, host memory is refused


class Args(dict):
    def __getattr__(self, k):
        return self[k]


def case(dtype=torch.bfloat16, R=3, Hq=4, Hk=2, D=128, NP=5, NR=2, MP=4, P=300, rot=64, fp4=False):
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32)
    u8 = lambda *s: torch.zeros(*s, dtype=torch.uint8)
    t = lambda *s: torch.zeros(*s, dtype=dtype)
    a = Args(k=t(R, Hk, D), v=t(R, Hk, D), page_table=i32(NR, MP), row_req=i32(R), row_pos=i32(R))
    if fp4:
        a.update(k_codes=u8(NP, 64, Hk, D // 2), k_scale=u8(NP, 64, Hk, D // 32), v_codes=u8(NP, 64, Hk, D // 2),
                 v_scale=u8(NP, 64, Hk, D // 32))
    else:
        a.update(k_cache=t(NP, 64, Hk, D), v_cache=t(NP, 64, Hk, D))
    a.update(status=i32(1), q=t(R, Hq, D), out_q=t(R, Hq, D), q_weight=t(D), k_weight=t(D), eps=1e-6, rope=torch.zeros(P, 2, rot // 2),
             rope_first=0)
    return a


def call(a, fp4=False):
    s = Stream()
    code = (m.idx_cache_append_fp4_async if fp4 else m.idx_cache_append_async)(**a, stream=s, raise_on_error=False)
    b = {k: v for k, v in a.items() if k != "status"}
    assert (m.idx_cache_append_fp4 if fp4 else m.idx_cache_append)(**b, stream=s, raise_on_error=False) == code
    return code


class Stream:
    cuda_stream = 0


needs_no_gpu = pytest.mark.skipif(torch.cuda.is_available(), reason="the accepted calls end at the missing device")


@needs_no_gpu
@pytest.mark.parametrize("fp4", [False, True])
def test_accepted(fp4):
    for kw in [{}, dict(dtype=torch.float16), dict(D=64), dict(D=256, rot=16), dict(R=0), dict(R=1)]:
        assert call(case(fp4=fp4, **kw), fp4) == 6, kw
    a = case(fp4=fp4)
    for drop in [("q", "out_q", "q_weight"), ("rope",), ("q_weight", "k_weight"), ("v", "v_codes" if fp4 else "v_cache") + (("v_scale",) if fp4 else ())]:
        assert call(Args({k: (None if k in drop else x) for k, x in a.items()}), fp4) == 6, drop
    a["out_q"] = a["q"]
    assert call(a, fp4) == 6
    a = case(fp4=fp4)
    wide = torch.zeros(3, 8, 128, dtype=torch.bfloat16)
    a.update(q=wide[:, :4], k=wide[:, 4:6], v=wide[:, 6:], q_weight=torch.zeros(128), k_weight=torch.zeros(128))
    assert call(a, fp4) == 6


@pytest.mark.parametrize("fp4", [False, True])
def test_refused_shapes_and_types(fp4):
    z = lambda *s, dtype=torch.bfloat16: torch.zeros(*s, dtype=dtype)
    kc = "k_codes" if fp4 else "k_cache"
    vc = "v_codes" if fp4 else "v_cache"
    bad = [dict(v=z(3, 1, 128)), dict(v=z(2, 2, 128)), dict(q=z(2, 4, 128)), dict(q=z(3, 4, 64)),
           dict(out_q=z(3, 5, 128)), dict(out_q=None), dict(q=None), dict(k=z(3, 2, 128, dtype=torch.float32)),
           dict(v=z(3, 2, 128, dtype=torch.float16)), dict(row_req=torch.zeros(2, dtype=torch.int32)),
           dict(row_pos=torch.zeros(3, dtype=torch.int64)), dict(eps=-1.0), dict(eps=float("nan")), dict(eps=float("inf")),
           dict(q_weight=z(64)), dict(k_weight=z(128, dtype=torch.float16)), dict(q_weight=torch.zeros(128)), dict(q=None, out_q=None),
           dict(rope=torch.zeros(300, 3, 32)), dict(rope=torch.zeros(300, 2, 4)), dict(rope=torch.zeros(300, 2, 72)),
           dict(rope=torch.zeros(0, 2, 32)), dict(rope_first=72), dict(rope_first=-8), dict(rope=torch.zeros(300, 2, 64)[:, :, :32]),
           dict(v=None), {vc: None}, dict(k=z(3, 2, 256)[..., ::2]), dict(q=z(3, 4, 132)[..., :128])]
    for change in bad:
        assert call(Args({**case(fp4=fp4), **change}), fp4) == INVALID, change.keys()
    for change in [dict(rope=torch.zeros(300, 2, 12)), dict(rope_first=4), dict(k=z(3, 2, 96), v=z(3, 2, 96))]:
        assert call(Args({**case(fp4=fp4), **change}), fp4) == UNSUPPORTED, change.keys()
    a = case(fp4=fp4, D=32, rot=16)
    assert call(a, fp4) == UNSUPPORTED
    a = case(fp4=fp4)
    x = a[kc]
    a[kc] = torch.zeros(5, 32, *x.shape[2:], dtype=x.dtype)
    assert call(a, fp4) != 6
    a = case(fp4=fp4)
    a[kc] = torch.zeros(5, 64, 3, x.shape[3], dtype=x.dtype)
    assert call(a, fp4) == INVALID
    if fp4:
        for name in ("k_scale", "v_scale"):
            a = case(fp4=True)
            a[name] = None
            assert call(a, True) == INVALID
            a[name] = torch.zeros(5, 64, 2, 8, dtype=torch.uint8)
            assert call(a, True) == INVALID
            a[name] = torch.zeros(5, 64, 2, 8, dtype=torch.uint8)[..., 2:6]     # not on the scales' own boundary
            assert call(a, True) == INVALID
        a = case(fp4=True)
        a["out_q"] = torch.zeros(3, 4, 64, dtype=torch.uint8)
        assert call(a, True) == INVALID                                          # codes without scales
        a["out_q_scale"] = torch.zeros(3, 4, 2, dtype=torch.uint8)
        assert call(a, True) == INVALID
        a = case(fp4=True)
        a["out_q_scale"] = torch.zeros(3, 4, 4, dtype=torch.uint8)
        assert call(a, True) == INVALID                                          # scales of 16-bit queries


@pytest.mark.parametrize("fp4", [False, True])
def test_refused_overlaps(fp4):
    kc, vc = ("k_codes", "v_codes") if fp4 else ("k_cache", "v_cache")
    a = case(fp4=fp4)
    a[vc] = a[kc]
    assert call(a, fp4) == INVALID
    a = case(fp4=fp4)
    a["out_q"] = torch.zeros(3, 1, 128, dtype=torch.bfloat16).expand(3, 4, 128)
    assert call(a, fp4) == INVALID                         # the heads of out_q share elements
    a = case(fp4=fp4)
    both = torch.zeros(4, 4, 128, dtype=torch.bfloat16)
    a["q"], a["out_q"] = both[:3], both[1:]
    assert call(a, fp4) == INVALID                         # overlaps q without being q
    a = case(fp4=fp4)
    a["k"] = a["out_q"][:, :2]
    assert call(a, fp4) == INVALID
    if not fp4:
        a = case()
        a["v"] = a["v_cache"][0, :3]
        assert call(a) == INVALID
        a = case()
        a["k_cache"] = a["k_cache"][:, :1].expand(5, 64, 2, 128)
        assert call(a) == INVALID


@needs_no_gpu
def test_queries_in_place_in_a_projection():
    a = case()
    wide = torch.zeros(3, 8, 128, dtype=torch.bfloat16)
    a.update(q=wide[:, :4], k=wide[:, 4:6], v=wide[:, 6:])
    a["out_q"] = a["q"]
    assert call(a) == 6
    a["k"] = wide[:, 3:5]
    assert call(a) == INVALID
    a["k"] = wide.flatten()[512:].as_strided((3, 2, 128), (512, 128, 1))
    assert call(a) == INVALID


@needs_no_gpu
def test_interleaved_places():
    a = case()
    both = torch.zeros(5, 2, 64, 2, 128, dtype=torch.bfloat16)
    a["k_cache"], a["v_cache"] = both[:, 0], both[:, 1]
    assert call(a) == 6
    a["v_cache"] = both.flatten()[128:128 + 5 * 2 * 64 * 2 * 128 - 128 * 2 * 64].as_strided((5, 64, 2, 128), (32768, 256, 128, 1), 128)
    assert call(a) == INVALID
    # codes and scales of a page one after the other
    a = case(fp4=True, Hk=1, R=3)
    page = torch.zeros(5, 2, 4352, dtype=torch.uint8)
    for i, x in enumerate("kv"):
        a[x + "_codes"] = page[:, i].as_strided((5, 64, 1, 64), (8704, 64, 64, 1), i * 4352)
        a[x + "_scale"] = page[:, i].as_strided((5, 64, 1, 4), (8704, 4, 4, 1), i * 4352 + 4096)
    assert call(a, True) == 6
    a["v_scale"] = page[:, 1].as_strided((5, 64, 1, 4), (8704, 4, 4, 1), 4352 + 4080)
    assert call(a, True) == INVALID


def test_packed_descriptors():
    """The descriptors that these calls pass, remembered by layout, are those of the struct; again, and at another
    address."""
    ts = [torch.zeros(7, 64, 64, dtype=torch.uint8), torch.zeros(5, dtype=torch.int32), torch.zeros(0, dtype=torch.int32),
          torch.zeros(3, 4)[:, ::2], torch.zeros(2, 3, 4, 5, 6), torch.zeros((), dtype=torch.float16), None,
          torch.zeros(6, 2, dtype=torch.float64), torch.zeros(9, 64, 64, dtype=torch.uint8)[2:], torch.zeros(3, 4).t()]
    for _ in range(2):
        for t, got in zip(ts, m._packed(ts)):
            assert got == (None if t is None else bytes(m._desc(t)))


def gather(a):
    s = Stream()
    code = m.idx_cache_gather_fp4_async(*a, torch.zeros(1, dtype=torch.int32), stream=s, raise_on_error=False)
    assert m.idx_cache_gather_fp4(*a, stream=s, raise_on_error=False) == code
    return code


def test_gather_refusals():
    u8 = lambda *s: torch.zeros(*s, dtype=torch.uint8)
    base = [u8(5, 64, 2, 64), u8(5, 64, 2, 4), u8(5, 64, 2, 64), u8(5, 64, 2, 4), torch.zeros(7, dtype=torch.int32),
            torch.zeros(7, 2, 128, dtype=torch.bfloat16), torch.zeros(7, 2, 128, dtype=torch.bfloat16)]
    if not torch.cuda.is_available():
        assert gather(base) == 6
        assert gather(base[:2] + [None, None] + base[4:6] + [None]) == 6
    for i, x in [(0, None), (1, None), (2, None), (3, None), (4, None), (5, None), (6, None), (1, u8(5, 64, 2, 2)), (2, u8(4, 64, 2, 64)),
                 (4, torch.zeros(7, 1, dtype=torch.int32)), (4, torch.zeros(7)), (5, torch.zeros(6, 2, 128, dtype=torch.bfloat16)),
                 (5, torch.zeros(7, 2, 128)), (6, torch.zeros(7, 2, 128, dtype=torch.float16)), (6, base[5]),
                 (5, torch.zeros(7, 1, 128, dtype=torch.bfloat16).expand(7, 2, 128))]:
        a = list(base)
        a[i] = x
        assert gather(a) == INVALID, i
    a = list(base)
    a[0] = u8(5, 64, 2, 48)
    assert gather(a) == UNSUPPORTED


def attend(a, slots=False):
    s = Stream()
    fn = m.idx_attn_selected_fp4 if slots else m.idx_attn_paged_fp4
    return fn(**a, stream=s, raise_on_error=False)


def attend_case(slots=False, dtype=torch.bfloat16, D=128, Hq=8, Hk=2, R=3, NP=5):
    u8 = lambda *s: torch.zeros(*s, dtype=torch.uint8)
    a = dict(q=torch.zeros(R, Hq, D, dtype=dtype), k_codes=u8(NP, 64, Hk, D // 2), k_scale=u8(NP, 64, Hk, D // 32),
             v_codes=u8(NP, 64, Hk, D // 2), v_scale=u8(NP, 64, Hk, D // 32), scale=0.1, out=torch.zeros(R, Hq, D, dtype=dtype),
             out_lse=torch.zeros(R, Hq))
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32)
    a.update(dict(slots=i32(R, 70)) if slots else dict(page_table=i32(2, 4), row_req=i32(R), row_start=i32(R), row_end=i32(R)))
    return a


@pytest.mark.parametrize("slots", [False, True])
def test_attention_refusals(slots):
    if not torch.cuda.is_available():
        for kw in [{}, dict(D=64), dict(D=256), dict(dtype=torch.float16), dict(R=0)]:
            assert attend(attend_case(slots, **kw), slots) == 6, kw
        a = attend_case(slots)
        a["v_codes"], a["v_scale"] = a["k_codes"], a["k_scale"]      # a latent cache: both are the same
        assert attend(a, slots) == 6
    u8 = lambda *s: torch.zeros(*s, dtype=torch.uint8)
    bad = [dict(k_scale=None), dict(v_scale=None), dict(k_codes=None), dict(k_scale=u8(5, 64, 2, 2)), dict(v_scale=u8(4, 64, 2, 4)),
           dict(v_codes=u8(5, 64, 1, 64)), dict(k_codes=u8(5, 64, 2, 128)), dict(k_scale=torch.zeros(5, 64, 2, 4)),
           dict(k_codes=torch.zeros(5, 64, 2, 64, dtype=torch.bfloat16)), dict(k_codes=u8(5, 64, 2, 72)[..., :64]),
           dict(k_scale=u8(5, 64, 2, 6)[..., :4]), dict(k_scale=u8(5, 64, 2, 4).flip(0)[1:]), dict(scale=0.0), dict(scale=float("nan")),
           dict(scale=float("inf")), dict(scale=-1.0), dict(out=torch.zeros(3, 8, 64, dtype=torch.bfloat16)), dict(out_lse=torch.zeros(3, 2)),
           dict(q=torch.zeros(3, 7, 128, dtype=torch.bfloat16), out=torch.zeros(3, 7, 128, dtype=torch.bfloat16))]
    bad += [dict(slots=None)] if slots else [dict(page_table=None), dict(row_end=torch.zeros(2, dtype=torch.int32))]
    for change in bad:
        assert attend({**attend_case(slots), **change}, slots) == INVALID, change.keys()
    a = attend_case(slots)
    a["out"] = a["q"]
    assert attend(a, slots) == INVALID
    a = attend_case(slots)
    a["out_lse"] = a["k_scale"].flatten()[:96].view(torch.float32).view(3, 8)
    assert attend(a, slots) == INVALID                               # the output lies in the scales
    a = attend_case(slots, D=96)
    assert attend(a, slots) == UNSUPPORTED
