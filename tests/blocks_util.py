"""Plain binary64 forms of the 8-bit blocks and of the AdamW step, with the error bounds that the GPU tests allow.

Bounds count roundings: U = 2^-24 is half a step of fp32.
"""
import numpy as np
import torch

from oracle.philox import philox4x32_10_np

U = 2.0 ** -24
HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}
BLOCK = 128


def blocks(n):
    return -(-n // BLOCK)


def e4m3(y):
    """The nearest e4m3 values (ties to even), magnitudes above 448 at 448."""
    y = np.asarray(y, np.float64)
    e = np.maximum(np.frexp(np.abs(y))[1] - 1, -6) - 3
    return np.clip(np.ldexp(np.rint(np.ldexp(y, -e)), e), -448.0, 448.0)


def scale_of(amax):
    """The scale of a block in fp32, NaN for one that is not finite."""
    s = np.maximum(amax.astype(np.float32) / np.float32(448), np.float32(2.0 ** -126))
    return np.where(np.isfinite(amax), s, np.float32(np.nan))


def in_units(v, amax):
    """Elements in units of their block's scale, the quotient rounded once to fp32 (binary64 before: 29 bits more)."""
    amax = amax.astype(np.float64)
    with np.errstate(invalid="ignore", divide="ignore", over="ignore"):
        y = np.where(amax >= 448 * 2.0 ** -126, v.astype(np.float64) * 448 / amax, v.astype(np.float64) * 2.0 ** 126)
    return np.where(np.isfinite(amax), y, 0.0).astype(np.float32)


def quantise(x, tile):
    """fp32 values [R, C] -> (code values [R, C], scales in the layout of the kind)."""
    x = np.asarray(x, np.float32)
    R, C = x.shape
    rows = BLOCK if tile else 1
    pad = np.zeros((-(-R // rows) * rows, blocks(C) * BLOCK), np.float32)
    pad[:R, :C] = x
    v = pad.reshape(pad.shape[0] // rows, rows, blocks(C), BLOCK)
    a = np.abs(v)
    amax = np.where(np.isnan(a).any(axis=(1, 3)), np.nan, a.max(axis=(1, 3)))
    s = scale_of(amax)
    y = e4m3(in_units(v, amax[:, None, :, None])).reshape(pad.shape)[:R, :C]
    return y, s if tile else s.T


def product(a, sa, b, sb, tile, base=None):
    """binary64 product of code values and scales (numpy), and the sum of the products' magnitudes."""
    K = a.shape[1]
    wa = a * np.repeat(sa.T, BLOCK, axis=1)[:, :K]
    s = np.repeat(sb, BLOCK, axis=0)[:b.shape[0]] if tile else sb.T
    wb = b * np.repeat(s, BLOCK, axis=1)[:, :K]
    want, size = wa @ wb.T, np.abs(wa) @ np.abs(wb).T
    return (want, size) if base is None else (want + base, size + np.abs(base))


def product_tol(size, K):
    # a block's sum in the matrix unit: at most one unit (2 U) per product; the product of the scales; one fused
    # multiply-add per block and what joins parts of the sum; the addition to the output
    return size * ((BLOCK * 2 + 2 + 2 * blocks(K) + 2) * U)


def words(n, high, step, index, seed):
    """The random word of every element."""
    i = np.arange(-(-n // 4))
    w = philox4x32_10_np(i & 0xFFFFFFFF, high, step & 0xFFFFFFFF, index, seed & 0xFFFFFFFF, seed >> 32)
    return np.stack(w, axis=1).reshape(-1)[:n].astype(np.int64)


def adamw(p, g, m, v, lr, step, b1, b2, eps, wd):
    """binary64 step on arrays; (value, m, v) and what each may be off by in fp32 arithmetic.

    m: b1 rounded, the product, the sum; 1 - b1 rounded, two products, the sum. v: the same with g twice. The change: m's
    own error, sqrt(v)'s (half of v's relative one and its own), the corrections (logarithm, product, expm1 and a
    reciprocal root of two units each), three operations; then the decay's product and the last rounding."""
    tm = U * (3 * np.abs(b1 * m) + 5 * np.abs((1 - b1) * g))
    m = b1 * m + (1 - b1) * g
    v = b2 * v + (1 - b2) * g * g
    tv = 7 * U * v
    root = np.sqrt(v)
    c1, c2 = 1 / (1 - b1 ** step), 1 / np.sqrt(1 - b2 ** step)
    den = root * c2 + eps
    change = m * c1 / den
    new = p - lr * (wd * p + change)
    tp = U * np.abs(new) + lr * (24 * U * np.abs(change) + tm * c1 / den + 4 * U * wd * np.abs(p))
    return (new, m, v), (tp, tm, tv)


def stochastic(x, tx, scale, h, least):
    """e4m3 values (in units of the scale) of magnitudes x after random rounding, and by how much each may be off: one step
    where x's error tx, the scale's and the sum's roundings leave open on which side of a whole number it falls."""
    y = x / scale
    e = np.maximum(np.frexp(y)[1] - 1, -6) - 3
    step = np.ldexp(1.0, e)
    t = y / step + (h + 0.5) / 65536
    off = (tx / scale) / step + 8 * U * t
    near = np.abs(t - np.rint(t)) <= off
    q = np.minimum(np.floor(t) * step, 448.0)
    if least:
        q = np.where(x > 0, np.maximum(q, 2.0 ** -9), q)
    return q, np.where(near, step, 0.0)


def per_block(x):
    pad = np.zeros(blocks(x.size) * BLOCK)
    pad[:x.size] = x
    return pad.reshape(-1, BLOCK)


def f64(t):
    return t.detach().double().cpu().numpy()
