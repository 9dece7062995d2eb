"""Plain forms of writing a paged cache for the tests, written from the formulas: the norm and the rotation in 64
bits with the bound that the kernel's arithmetic gives, the same in 32 bits rounding by rounding, and the 4-bit form.

Bounds, in units of 2^-24 relative.  What becomes 4 bits is rounded where the documented order says: the sum of squares,
the addition of eps (both under a root: half), the root, the reciprocal, the product with x and that with the weight: 5 of
a normed element.  A rotation adds a rounded product each (6 of |a cos| and of |b sin|) and the rounding of their sum: 7
(|a cos| + |b sin|) at most.  What stays in 16 bits sums the squares (all positive) in fp32, 8 a lane and then up to 32
lanes: at most 13 roundings; one with eps, half of these 14 in the root; a reciprocal root of 2 units in the last place (4);
two products: 13 of a normed element, 15 (|a cos| + |b sin|) of a rotated one.  The cosines and sines are inputs.  A 16-bit
output adds u |y| (fp16 below its normal range: 2^-25).
"""
import numpy as np

U = {"bfloat16": 2.0 ** -8, "float16": 2.0 ** -11}
E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def _pairs(rot, first, pairs):
    i = np.arange(rot // 2)
    return (first + 2 * i, first + 2 * i + 1) if pairs else (first + i, first + rot // 2 + i)


def turned64(x, weight, eps, cos, sin, first, pairs, four=True):
    """x [R, H, D] (float64 of the inputs), weight [D] or None, cos and sin [R, rot / 2] or None ->
    y and the bound of the kernel's error before the last rounding (`four`: to 4 bits)."""
    x = np.asarray(x, dtype=np.float64)
    y, units = x.copy(), np.zeros_like(x)
    if weight is not None:
        y = x / np.sqrt((x * x).mean(-1, keepdims=True) + float(np.float32(eps))) * weight
        units = (5 if four else 13) * np.abs(y)
    if cos is not None:
        a, b = _pairs(2 * cos.shape[1], first, pairs)
        c, s = cos[:, None].astype(np.float64), sin[:, None].astype(np.float64)
        ya, yb = y[..., a], y[..., b]
        units[..., a] = (7 if four else 15) * (np.abs(ya * c) + np.abs(yb * s))
        units[..., b] = (7 if four else 15) * (np.abs(yb * c) + np.abs(ya * s))
        y[..., a], y[..., b] = ya * c - yb * s, yb * c + ya * s
    return y, units * 2.0 ** -24 * (1 + 1e-6) + 1e-44


def turned32(x, weight, eps, cos, sin, first, pairs):
    """The same with every product and sum rounded to 32 bits in the documented order, and the sum of squares once."""
    f = np.float32
    y = np.asarray(x, dtype=f)
    if weight is not None:
        total = (y.astype(np.float64) ** 2).sum(-1, keepdims=True).astype(f)
        r = f(1) / np.sqrt(total / f(y.shape[-1]) + f(eps))
        y = (y * r) * np.asarray(weight, dtype=f)
    if cos is not None:
        a, b = _pairs(2 * cos.shape[1], first, pairs)
        c, s = cos[:, None].astype(f), sin[:, None].astype(f)
        out = y.copy()
        out[..., a], out[..., b] = y[..., a] * c - y[..., b] * s, y[..., b] * c + y[..., a] * s
        y = out
    assert y.dtype == f
    return y


def quantise(x):
    """x [.., D] float64 or float32 (finite) -> code indices (0..15) [.., D], scale bytes [.., D / 32]."""
    b = np.asarray(x, dtype=np.float64).reshape(*x.shape[:-1], -1, 32)
    top = np.abs(b).max(-1, keepdims=True)
    e = np.full(top.shape, -127)
    for k in range(-127, 128):            # the smallest e whose range holds the block
        e = np.where(top > 6 * 2.0 ** k, k + 1, e)
    y = b / 2.0 ** e
    d = np.abs(np.abs(y)[..., None] - E2M1)
    near = d.min(-1, keepdims=True)
    idx = np.argmax((d == near) & (np.arange(8) % 2 == 0), -1)       # of two that are equally near the even one
    idx = np.where(((d == near) & (np.arange(8) % 2 == 0)).any(-1), idx, np.argmax(d == near, -1))
    return (idx + 8 * np.signbit(y)).reshape(x.shape), (e[..., 0] + 127).astype(np.uint8)


def unpack(codes):
    """Bytes [.., D / 2] -> code indices [.., D]."""
    c = np.asarray(codes)
    return np.stack([c & 15, c >> 4], -1).reshape(*c.shape[:-1], 2 * c.shape[-1])


def values(idx, scale):
    """Code indices [.., D] and scale bytes [.., D / 32] -> the numbers (float64; 255: NaN)."""
    v = E2M1[idx & 7] * np.where(idx >= 8, -1.0, 1.0)
    s = np.where(scale == 255, np.nan, 2.0 ** (scale.astype(np.float64) - 127))
    return (v.reshape(*idx.shape[:-1], idx.shape[-1] // 32, 32) * s[..., None]).reshape(idx.shape)


def check_codes(idx, scale, y, bound):
    """Codes and scales that a result within `bound` of y may have."""
    shape = idx.shape
    b, d = y.reshape(*shape[:-1], -1, 32), bound.reshape(*shape[:-1], -1, 32)
    s = 2.0 ** (scale.astype(np.float64) - 127)[..., None]
    low, high = (np.abs(b) - d).max(-1, keepdims=True), (np.abs(b) + d).max(-1, keepdims=True)
    assert (low <= 6 * s).all(), "a block is cut off"
    assert ((high > 3 * s) | (scale[..., None] == 0)).all(), "a scale is too large"
    got = (E2M1[idx & 7] * np.where(idx >= 8, -1.0, 1.0)).reshape(b.shape) * s
    near = np.abs(b[..., None] / s[..., None] - np.concatenate([E2M1, -E2M1])).min(-1) * s
    over = np.abs(got - b) - near - 2 * d
    assert (over <= 0).all(), float(over.max())


def to64(t):
    return t.detach().double().cpu().numpy()
