"""Attention over a paged cache in 64 bits (numpy), with bounds on the rounding
error of an evaluation in fp32, and the cache's append.

U = 2^-24, half a step of fp32.  With s_j the scores, A_j = |scale| sum |q_d k_jd|,
P_j the weights (they sum to 1) and n the number of keys:

* a score: N products (exact for bf16) added one after another, at most 2 U of the
  sum of their sizes for each addition (a matrix unit may cut instead of rounding):
  2 (N + 1) U A_j; the scale with log2 e, the subtraction of the maximum and the
  exponential's argument: 3 U (|s_j| + max |s|) more, in the exponent; so the weight is
  off by that share of itself, and by 2 U more from the exponential;
* the running maximum changes at most n times, each time everything is scaled: the
  factor cancels between sum and products, its two roundings (2 U each) do not;
* sums of n terms: 2 n U of the sum of their sizes;
* bf16: a weight is rounded before the product with the values, half a step of bf16
  (2^-8 of itself), though not in the sum;
* joining waves and pieces: 10 U.
"""
import numpy as np

U = 2.0 ** -24


def attend(q, k, v, pos, scale, window, half):
    """q [n, N] at positions pos [n], k, v [S, N] at positions 0 .. S-1 (rows
    of keys that lie on no page hold NaN in `k` and are not seen): out [n, N], lse
    [n] and their bounds.  half: half a step of the weights' type (0 for fp32)."""
    n, N = q.shape
    S = k.shape[0]
    out, eout = np.zeros((n, N)), np.zeros((n, N))
    lse, else_ = np.full(n, -np.inf), np.zeros(n)
    j = np.arange(S)
    there = ~np.isnan(k).all(-1) if S else np.zeros(0, bool)
    for i in range(n):
        seen = there & (j <= pos[i])
        if window:
            seen &= j > pos[i] - window
        kk, vv = k[seen], v[seen]
        if len(kk) == 0:
            continue
        s = scale * (kk @ q[i])
        A = abs(scale) * (np.abs(kk) @ np.abs(q[i]))
        m = s.max()
        w = np.exp(s - m)
        l = w.sum()
        P = w / l
        out[i] = P @ vv
        lse[i] = m + np.log(l)
        e = 2 * (N + 1) * U * A + 3 * U * (np.abs(s) + np.abs(s).max()) + 2 * U
        e = np.expm1(e)
        c = len(kk)
        el = (P * e).sum() + (4 * c + 10) * U
        eout[i] = (P * (e + half + el)) @ np.abs(vv) + (6 * c + 10) * U * (P @ np.abs(vv))
        else_[i] = 1.01 * el + 4 * U * (1 + abs(lse[i]) + abs(m))
    return out, lse, eout, else_


def turn(x, pos, freqs, interleaved):
    """R(pos) x for x [..., N], pos broadcast over the leading axes; and a bound: cos
    and sin are off by at most 8 U (the angle's fraction of a turn is rounded once, pi U,
    the functions are good to two steps), two products and an addition round: 10 U of both
    elements."""
    if freqs is None:
        return x, np.zeros_like(x)
    ang = np.asarray(pos, np.float64)[..., None] * freqs.astype(np.float64)
    c, s = np.cos(ang), np.sin(ang)
    n = len(freqs)
    y, e = x.copy(), np.zeros_like(x)
    a, b = (slice(0, 2 * n, 2), slice(1, 2 * n, 2)) if interleaved else (slice(0, n), slice(n, 2 * n))
    p, q = x[..., a], x[..., b]
    y[..., a], y[..., b] = p * c - q * s, p * s + q * c
    e[..., a] = e[..., b] = 10 * U * (np.abs(p) + np.abs(q))
    return y, e
