"""Plain 64-bit attention and eviction for the tests, written from the formulas, and the
error bounds that the kernels' arithmetic gives.

Bounds.  The kernel forms a score as a sum of D exact 16-bit products accumulated in fp32
(at most D roundings of 2^-23 relative to the sum of magnitudes), scales it and takes a
base-2 exponential (relative error below 2^-21): with e_s = (D + 8) 2^-23 scale sum |q k|
at most over the row's positions, every softmax weight p has a relative error of at most
e_p = 2 e_s + 2^-20 after the division by the sum.  The product with the values rounds p to
the inputs' type (unit roundoff u; below the type's normal range an absolute 2^-25 for
fp16) and the result to the same type:
    |out - exact| <= u |exact| + (u + e_p + n 2^-24) sum_j p_j |v_j| + n 2^-25 max |v| [fp16].
lse: e_s + 2^-20 + 2^-22 |lse|.  A position's weight: the sum over rows and heads of p e_p,
and 2^-22 of the total for its additions.
"""
import math

import numpy as np

U = {"bfloat16": 2.0 ** -8, "float16": 2.0 ** -11}


def _u(t):
    return U[str(t.dtype).replace("torch.", "")]


def attend(q, k, v, scale):
    """One row: q [Hq, D], k, v [n, Hk, D] in any type -> out, lse, p [Hq, n], and the bounds
    of out and lse and the weights' relative bound, in float64."""
    import torch
    u, f16 = _u(q), q.dtype == torch.float16
    q, k, v = q.double(), k.double(), v.double()
    Hq, D = q.shape
    n, Hk = k.shape[0], k.shape[1]
    if n == 0:
        z = torch.zeros(Hq, D, dtype=torch.float64, device=q.device)
        return (z, torch.full((Hq,), -math.inf, dtype=torch.float64, device=q.device),
                torch.zeros(Hq, 0, dtype=torch.float64, device=q.device), z, torch.zeros_like(z[:, 0]), 0.0)
    head = torch.arange(Hq, device=q.device) // (Hq // Hk)
    kh, vh = k[:, head], v[:, head]                    # [n, Hq, D]
    s = torch.einsum("hd,nhd->hn", q, kh) * scale
    m = s.max(1, keepdim=True).values
    e = torch.exp(s - m)
    l = e.sum(1, keepdim=True)
    p = e / l
    out = torch.einsum("hn,nhd->hd", p, vh)
    lse = (m + torch.log(l))[:, 0]
    mag = torch.einsum("hd,nhd->hn", q.abs(), kh.abs()).max(1).values * scale
    es = (D + 8) * 2.0 ** -23 * mag
    ep = 2 * es + 2.0 ** -20
    a = torch.einsum("hn,nhd->hd", p, vh.abs())
    bound = u * out.abs() + (u + ep[:, None] + n * 2.0 ** -24) * a + (n * 2.0 ** -25 * v.abs().max() if f16 else 0.0) + 1e-30
    return out, lse, p, bound, es + 2.0 ** -20 + 2.0 ** -22 * lse.abs(), ep


def check_rows(q, out, lse, rows, scale):
    """rows[r] = (k, v) of row r's positions, in order."""
    import torch
    for r, (k, v) in enumerate(rows):
        want, wl, _, bo, bl, _ = attend(q[r], k, v, scale)
        err = (out[r].double() - want).abs()
        assert bool((err <= bo).all()), (r, float((err - bo).max()), float(err.max()))
        if lse is not None:
            if k.shape[0] == 0:
                assert bool(torch.isneginf(lse[r]).all()), r
            else:
                el = (lse[r].double() - wl).abs()
                assert bool((el <= bl).all()), (r, float(el.max()))


def order_key(w):
    """The selection's order as sortable integers (larger is kept first)."""
    b = np.asarray(w, dtype=np.float32).view(np.uint32).astype(np.int64)
    key = np.where(b >= 2 ** 31, 2 ** 32 - 1 - b, b + 2 ** 31)
    return np.where(np.isnan(w), 0, key)


def keep_positions(w, n, budget, first, last):
    """Kept positions of one request of length n with weights w."""
    if n <= budget:
        return list(range(n))
    mid = list(range(first, n - last))
    key = order_key(np.asarray(w)[:n])
    mid.sort(key=lambda i: (-int(key[i]), i))
    return sorted(list(range(first)) + mid[: budget - first - last] + list(range(n - last, n)))
