"""Plain 64-bit attention over a cache in 4 bits for the tests, and the error bounds of the kernels' arithmetic.

Bounds.  As in tests/attn_ref.py, with what the 4-bit form changes.  Codes times a power of two are exact in fp16, so
a score is a sum of D exact products accumulated in fp32 (D + 8 roundings of 2^-23 of the sum of magnitudes at most);
blocks of keys below 2^-26 of the largest scale near them may count as 0, which takes 6 * 2^(E - 127 - 27) from an
element at most (E the largest scale byte): 6 * 2^(E - 154) scale |q|_1 of a score.  bf16 queries keep all bits down to
2^-38 of the head's largest, and lose 2^-39 of it below: D 2^-39 max |q| max |k| scale of a score.  With e_s the sum
of these a weight is off by e_p = 2 e_s + 2^-20 relative.  Weights are rounded to fp16 (2^-11; below 2^-24 of the
largest 2^-35 each), values' small blocks cost another 6 * 2^(E - 154), and the result is rounded to q's type (u):
    |out - exact| <= u |out| + (2^-11 + e_p + n 2^-24) sum p |v| + n 2^-35 max |v| + 6 * 2^(E - 154) + sub
(sub: half the smallest step of the type, for results below its normal numbers: fp16 2^-25, bf16 2^-134, as its
exponents end at -126 and 7 bits follow: steps of 2^-133.)
lse: e_s + 2^-20 + 2^-22 |lse|.
"""
import math

U = {"bfloat16": 2.0 ** -8, "float16": 2.0 ** -11}


def values(codes, scales):
    """Codes u8 [.., D / 2] and scales u8 [.., D / 32] -> the numbers in 64 bits [.., D] (255: NaN)."""
    import torch
    t = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], dtype=torch.float64, device=codes.device)
    t = torch.cat([t, -t])
    c = codes.long()
    x = torch.stack([t[c & 15], t[c >> 4]], -1).flatten(-2)
    s = torch.exp2(scales.double() - 127)
    s = torch.where(scales == 255, torch.nan, s)
    return (x.unflatten(-1, (scales.shape[-1], 32)) * s[..., None]).flatten(-2)


def attend(q, k, v, scale, ek, ev):
    """One row: q [Hq, D], k and v [n, Hk, D] in 64 bits, ek and ev the largest scale bytes near -> out, lse, bounds."""
    import torch
    u = U[str(q.dtype).replace("torch.", "")]
    sub = 2.0 ** -25 if q.dtype == torch.float16 else 2.0 ** -134
    q = q.double()
    Hq, D = q.shape
    n, Hk = k.shape[0], k.shape[1]
    if n == 0:
        z = torch.zeros(Hq, D, dtype=torch.float64, device=q.device)
        return z, torch.full((Hq,), -math.inf, dtype=torch.float64, device=q.device), z, torch.zeros_like(z[:, 0])
    head = torch.arange(Hq, device=q.device) // (Hq // Hk)
    kh, vh = k[:, head], v[:, head]
    s = torch.einsum("hd,nhd->hn", q, kh) * scale
    m = s.max(1, keepdim=True).values
    e = torch.exp(s - m)
    l = e.sum(1, keepdim=True)
    p = e / l
    out, lse = torch.einsum("hn,nhd->hd", p, vh), (m + torch.log(l))[:, 0]
    mag = torch.einsum("hd,nhd->hn", q.abs(), kh.abs()).max(1).values * scale
    es = (D + 8) * 2.0 ** -23 * mag + 6 * 2.0 ** (ek - 154) * scale * q.abs().sum(1)
    es = es + D * 2.0 ** -39 * scale * q.abs().max(1).values * k.abs().max()
    ep = 2 * es + 2.0 ** -20
    a = torch.einsum("hn,nhd->hd", p, vh.abs())
    bound = u * out.abs() + (2.0 ** -11 + ep[:, None] + n * 2.0 ** -24) * a * (1 + u) + n * 2.0 ** -35 * v.abs().max()
    return out, lse, bound + 6 * 2.0 ** (ev - 154) + sub * (1 + u), es + 2.0 ** -20 + 2.0 ** -22 * lse.abs()


def check_rows(q, out, lse, rows, scale):
    """rows[r] = (key codes, key scales, value codes, value scales) of row r's positions, in order."""
    import torch
    some = [r for r in rows if r[0].shape[0]]
    ek, ev = (max([int(r[i].max()) for r in some], default=0) for i in (1, 3))
    for r, (kc, ks, vc, vs) in enumerate(rows):
        want, wl, bo, bl = attend(q[r], values(kc, ks), values(vc, vs), scale, ek, ev)
        err = (out[r].double() - want).abs()
        assert bool((err <= bo).all()), (r, float((err - bo).max()), float(err.max()))
        if lse is not None:
            if kc.shape[0] == 0:
                assert bool(torch.isneginf(lse[r]).all()), r
            else:
                el = (lse[r].double() - wl).abs()
                assert bool((el <= bl).all()), (r, float(el.max()), float((el - bl).max()))
