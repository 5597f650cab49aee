"""A bound for the fp32 attention over a key/value cache that 16 significand bits do not meet.

Sums of many products are as loose as they are long, so these inputs have short ones: a query has
one element that is not zero, so that a score is one product, and a row sees few keys.  What is
left, per row of n keys, with s a score (times scale, in nats), m the row's largest:

  * a score: the factor scale * log2(e) is rounded twice, the scaled query or the scaled score
    once; the product once, or on the tensor cores cut off below 2^-22 of it (six of nine terms of
    three parts each) and rounded off (up to 2^-23) by the last addition, the other terms being
    2^-7 of it: 2^-21 |s| together (2^-22 + 1.1 2^-23 + 3 2^-24 = 1.93 2^-22);
  * its distance to the reference, one rounding, and the reference may lie 8 binary steps below m:
    2^-24 (|s - m| + 6);
  * the exponential, 2^-22 of it: together r = 2^-21 |s| + 2^-24 (|s - m| + 6) + 2^-22 of a weight;
  * the sum of n weights: n 2^-24; a normalised weight is off by r + sum_j w_j r_j + n 2^-24;
  * the output: n products added up, each addition up to 2^-23 on the tensor cores (1.1 times, for
    the terms of small parts), its terms cut off below 2^-22: (1.1 n 2^-23 + 2^-22) sum_j w_j |v_j|;
  * joining what warps, blocks and splits have, and the division: an exponential, a product and an
    addition each, 2^-22 + 2^-23 twice over (block, then splits), 2^-23 for 1 / l times the output:
    under 2^-20;
  * a key's weights from the rows' log-sums: the log-sum, log2(l) and its addition to the reference
    rounded, and the subtraction once more: 2^-23 (|s| + |m| + log n + 8) instead of the division.
"""
import numpy as np


def full(x):
    """fp32 values whose last eight significand bits are ones: what goes with them is no accident."""
    return (np.asarray(x, np.float32).view(np.uint32) | np.uint32(0xff)).view(np.float32)


def one_hot_queries(rng, shape):
    """[..., D] queries with one element each, from 0.5 to 2."""
    q = np.zeros(shape, np.float32)
    at = rng.integers(0, shape[-1], shape[:-1])
    x = full(rng.uniform(0.5, 2.0, shape[:-1]) * rng.choice([-1, 1], shape[:-1]))
    np.put_along_axis(q, at[..., None], x[..., None], -1)
    return q


def cut(x, bits):
    """fp32 values cut to so many significand bits."""
    u = np.asarray(x, np.float32).view(np.uint32)
    return (u & np.uint32(0xffffffff << (24 - bits) & 0xffffffff)).view(np.float32)


def head(q, k, v, see, scale):
    """One head: q [Nq, D], k, v [n, D], see [Nq, n].  Output, its bound; the keys' weights, their bound."""
    q, k, v = (np.asarray(x, np.float64) for x in (q, k, v))
    any_ = see.any(1, keepdims=True)
    s = np.where(see, scale * (q @ k.T), -np.inf)
    m = np.where(any_, s.max(1, keepdims=True, initial=-np.inf), 0.0)
    w = np.exp(s - m)
    w /= np.where(any_, w.sum(1, keepdims=True), 1.0)
    n = see.sum(1, keepdims=True)
    a = np.where(see, np.abs(s), 0.0)
    r = np.where(see, 2.0 ** -21 * a + 2.0 ** -24 * (np.where(see, np.abs(s - m), 0.0) + 6) + 2.0 ** -22, 0.0)
    off = r + (w * r).sum(1, keepdims=True) + n * 2.0 ** -24
    o, size = w @ v, w @ np.abs(v)
    tol = (w * off) @ np.abs(v) + (1.1 * n * 2.0 ** -23 + 2.0 ** -22 + 2.0 ** -20) * size + 2.0 ** -24 * np.abs(o) + 1e-30
    wtol = w * (off + 2.0 ** -23 * (a + np.abs(m) + np.log(np.maximum(n, 1)) + 8) + 2.0 ** -22)
    return o, tol, w.sum(0), wtol.sum(0)


def call(q, k, v, lens, scale, visible, kp=None, vp=None, causal=True):
    """All heads.  visible(n) gives [Nq, S] truth values of a sequence of n tokens.  Outputs, bounds,
    the sums of the own keys' weights, their bounds."""
    B, H, Nq, D = q.shape
    Hk, S = k.shape[1:3]
    P = 0 if kp is None else kp.shape[1]
    o, tol = np.zeros((B, H, Nq, D)), np.zeros((B, H, Nq, D))
    got, wtol = np.zeros((B, Hk, S)), np.zeros((B, Hk, S))
    for b in range(B):
        before = np.ones((Nq, P), bool)
        if causal:
            before &= (lens[b] - Nq + np.arange(Nq) >= 0)[:, None]
        see = np.concatenate([before, visible(lens[b])], 1)
        for h in range(H):
            hk = h * Hk // H
            kk, vv = (x[b, hk] if P == 0 else np.concatenate([y[hk], x[b, hk]]) for x, y in ((k, kp), (v, vp)))
            o[b, h], tol[b, h], w, wt = head(q[b, h], kk, vv, see, scale)
            got[b, hk] += w[P:]
            wtol[b, hk] += wt[P:]
    return o, tol, got, wtol + (H // Hk * Nq + 2) * 2.0 ** -24 * got


# B, H, Hk, Nq, P, S, D, window, sinks, lens: few rows and many (causal windows, prefixes, whole caches)
SINK = [(3, 8, 2, 1, 0, 500, 64, 7, 2, [500, 300, 3]), (2, 6, 6, 4, 0, 90, 128, 5, 1, [90, 2]),
        (2, 64, 64, 300, 0, 310, 64, 8, 2, [310, 200]), (1, 64, 32, 260, 0, 260, 128, 6, 0, [260])]
PREFIX = [(4, 8, 2, 1, 5, 6, 128, None, 0, [6, 1, 0, 4]), (2, 64, 64, 130, 5, 6, 64, None, 0, [6, 2]),
          (1, 64, 64, 130, 3, 9, 128, None, 0, [8])]
CACHE = [(3, 8, 2, 1, 0, 12, 64, None, 0, [12, 1, 0]), (2, 12, 2, 1, 0, 9, 128, None, 0, [9, 5]),
         (2, 8, 2, 12, 0, 12, 64, None, 0, [12, 5]), (1, 4, 1, 10, 0, 11, 128, None, 0, [11])]
SCALE = 2.0


def inputs(seed, B, H, Hk, Nq, P, S, D):
    rng = np.random.default_rng(seed)
    draw = lambda *shape: full(rng.normal(size=shape))  # noqa: E731
    return [one_hot_queries(rng, (B, H, Nq, D)), draw(B, Hk, S, D), draw(B, Hk, S, D), draw(Hk, P, D), draw(Hk, P, D)]
