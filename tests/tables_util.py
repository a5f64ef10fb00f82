"""Plain binary64 forms of the vocabulary-side operators (token scores, their gradient, the 4-bit head, the embedding
and its gradient), with the error bounds that the GPU tests allow.

Bounds count roundings. u = 2^-24 is half a step of fp32; an output type rounds once more by half of its step
(2^-24 fp32, 2^-8 bf16).
"""
import numpy as np
import torch

IGNORE = -100
U = 2.0 ** -24
HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}


def order(x):
    """Indices of a row by (value descending, index ascending), -0 equal to +0."""
    return np.argsort(-(x + 0.0), kind="stable")


def score_row(x, t, T, n):
    """(status, logprob, entropy, rank, alt_idx, alt_lp, row_max, row_logsum) of a row of float64 logits."""
    idx = np.full(n, -1, np.int64)
    alt = np.full(n, np.nan)
    if t == IGNORE:
        return 0, 0.0, 0.0, -1, idx, alt, 0.0, 0.0
    m = x.max()                                   # NaN if there is one
    if not np.isfinite(m):
        return 4, np.nan, np.nan, -1, idx, alt, np.nan, np.nan
    if not 0 <= t < len(x) or not np.isfinite(T):
        return 1, np.nan, np.nan, -1, idx, alt, np.nan, np.nan
    T = T if T > 0 else 1.0
    s = (x - m) / T
    e = np.exp(s)
    S = e.sum()
    ls = np.log(S)
    A = np.where(e > 0, e * np.where(np.isfinite(s), s, 0.0), 0.0).sum()
    rank = int(((x > x[t]) | ((x == x[t]) & (np.arange(len(x)) < t))).sum())
    o = order(x)[:n]
    o = o[x[o] > -np.inf]
    idx[:len(o)] = o
    alt[:len(o)] = np.minimum(s[o] - ls, 0.0)
    return 0, min(s[t] - ls, 0.0), max(ls - A / S, 0.0), rank, idx, alt, m, ls


# log S: every term carries its exponential's error (4 u), the rounding of its exponent (3 u |s|, and terms that weigh
# have |s| up to about 30) and at most 64 + 8 additions of positive terms in fp32
LOGSUM_TOL = (4 + 3 * 30 + 72) * U


def logprob_tol(lp):
    return LOGSUM_TOL + 4 * U * np.abs(np.where(np.isfinite(lp), lp, 0.0))


def entropy_tol(ls):
    # log S - A / S, |A / S| <= log S: twice the relative error of a sum, and log S's own
    return LOGSUM_TOL * (2 + 2 * abs(ls))


def grad_row(x, t, T, g, h):
    """The gradient of g * logprob + h * entropy for a row of float64 logits (zeros for an ignored row), and the sum
    of the magnitudes that a rounding error is relative to."""
    if t == IGNORE:
        return np.zeros(len(x)), np.zeros(len(x))
    T = T if T > 0 else 1.0
    s = (x - x.max()) / T
    e = np.exp(s)
    ls = np.log(e.sum())
    p = e / e.sum()
    lp = np.where(p > 0, s - ls, 0.0)
    H = -(p * lp).sum()
    d = -p * (g + h * (lp + H))
    size = p * (abs(g) + abs(h) * (np.abs(lp) + H)) * (1 + np.abs(lp))
    d[t] += g
    size[t] += abs(g)
    return d / T, size / T


# p carries log S's error, the exponential's and its exponent's roundings (relative to 1 + |log p|)
GRAD_REL = LOGSUM_TOL + 16 * U


def unpack(codes):
    q = np.empty((codes.shape[0], codes.shape[1] * 2), np.float64)
    q[:, 0::2] = codes & 15
    q[:, 1::2] = codes >> 4
    return q


def head(hidden, codes, scales, zeros, group):
    """float64 logits and the sum of the products' magnitudes."""
    q = unpack(codes)
    z = np.full(scales.shape, 8.0) if zeros is None else zeros.astype(np.float64)
    w = (q - np.repeat(z, group, axis=1)) * np.repeat(scales, group, axis=1)
    return hidden @ w.T, np.abs(hidden) @ np.abs(w).T


def head_tol(size, group, groups, terms):
    # sums of a group in the matrix unit: at most one unit (2 u) per product of every term; then one fused
    # multiply-add per group; what three bf16 terms leave of an fp32 value is below 2 u
    return size * ((group * terms * 2 + groups + 2 + (2 if terms == 3 else 0)) * U)


def embed_grad(token, dout, V, scale, base=None):
    total = np.zeros((V, dout.shape[1])) if base is None else base.astype(np.float64).copy()
    size = np.zeros_like(total)
    count = np.zeros(V)
    ok = (token >= 0) & (token < V)
    np.add.at(total, token[ok], dout[ok] * scale)
    np.add.at(size, token[ok], np.abs(dout[ok]) * abs(scale))
    np.add.at(count, token[ok], 1)
    if base is not None:
        size += np.abs(base)
    return total, size * (count + 4)[:, None] * U


def f64(t):
    return t.detach().double().cpu().numpy()
