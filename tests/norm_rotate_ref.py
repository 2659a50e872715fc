"""Norm and rotation of head vectors in 64 bits (numpy), with bounds on the
rounding error of an fp32 evaluation.

U = 2^-24, half a step of fp32.  What one evaluation may lose:

* rstd: the sum of N <= 256 squares in a tree of at most 8 successive and 5
  exchanged additions, the division by N, eps: (8 + 5 + 3) U of a sum of
  positive terms, halved by the root, and the root to a step: 10 U;
* n * w: three products, so y before the turn is off by 13 U relative;
* cos and sin: the fraction of a turn is at most 1/2 and is rounded once (pi U
  as an angle), the functions are good to 2 steps (4 U): 8 U absolute;
* a turn of (u, v): (8 + 2) U (|u| + |v|) on top of what u and v carry.
"""
import numpy as np

U = 2.0 ** -24


def _angles(pos, freqs, interleaved, N):
    """cos, sin per element [b, L, 1, N] and the partner's index and sign."""
    R = 2 * len(freqs)
    ang = pos.astype(np.float64)[..., None] * freqs.astype(np.float64)
    b, L = pos.shape
    c, s = np.ones((b, L, 1, N)), np.zeros((b, L, 1, N))
    partner, sign = np.arange(N), np.zeros(N)
    for j in range(R // 2):
        p, q = (2 * j, 2 * j + 1) if interleaved else (j, j + R // 2)
        c[:, :, 0, p] = c[:, :, 0, q] = np.cos(ang[..., j])
        s[:, :, 0, p] = s[:, :, 0, q] = np.sin(ang[..., j])
        partner[p], partner[q], sign[p], sign[q] = q, p, -1.0, 1.0
    return c, s, partner, sign


def forward(x, w, pos, freqs, eps, interleaved):
    """(y, bound) for x [b, L, H, N]."""
    N = x.shape[-1]
    rstd = 1.0 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    u = x * rstd * (1.0 if w is None else w)
    if freqs is None:
        return u, 13 * U * np.abs(u)
    c, s, partner, sign = _angles(pos, freqs, interleaved, N)
    y = u * c + sign * u[..., partner] * s
    turned = sign != 0
    both = np.abs(u) + np.where(turned, np.abs(u[..., partner]), 0.0)
    return y, np.where(turned, 23.0, 13.0) * U * both


def backward(x, w, pos, freqs, eps, interleaved, dy, adds):
    """dict of dx, dw and their bounds edx, edw; adds: successive fp32
    additions behind one element of dw."""
    N = x.shape[-1]
    rstd = 1.0 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    n = x * rstd
    w1 = np.ones(N) if w is None else w
    v, P = dy, np.zeros_like(dy)
    if freqs is not None:
        c, s, partner, sign = _angles(pos, freqs, interleaved, N)
        v = dy * c - sign * dy[..., partner] * s
        P = np.where(sign != 0, np.abs(dy) + np.abs(dy[..., partner]), 0.0)
    ev = 10 * U * P
    wv = w1 * v
    m = (wv * n).mean(-1, keepdims=True)
    dx = rstd * (wv - n * m)
    em = (np.abs(w1) * ev * np.abs(n)).mean(-1, keepdims=True) + 30 * U * np.abs(wv * n).mean(-1, keepdims=True)
    edx = rstd * (np.abs(w1) * ev + 3 * U * np.abs(wv) + np.abs(n) * em + 14 * U * np.abs(n * m)) + 12 * U * np.abs(dx)
    t = v * n
    et = ev * np.abs(n) + 12 * U * np.abs(t)
    return dict(dx=dx, edx=edx, dw=t.sum((0, 1, 2)), edw=et.sum((0, 1, 2)) + adds * U * np.abs(t).sum((0, 1, 2)))
