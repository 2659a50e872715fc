"""The gated linear recurrence in 64 bits, token by token (numpy), with a bound
on the rounding error of an fp32 evaluation carried along.

U = 2^-24 is half a step of fp32.  What one fp32 evaluation may lose, in U:

* a sigmoid: the exponent's argument is one product-sum (its error grows with
  |v|), exp2 and the reciprocal are good to a step (2 U) each, one addition:
  (|v| + 6) U relative;
* the decay: exp2 to a step plus |log a| times the error of A * s;
* beta = sqrt(1 - a^2): the root to a step and half the relative error of
  1 - a^2, which is that of log a near a = 1 and 8 U elsewhere;
* every fma of the recurrence: one rounding of its result.  Composing maps of
  token groups in a tree adds at most as many roundings of the same products
  as there are levels; 8 U per token covers both.

What such a rounding is relative to: composed maps hold partial sums.  For
h_2 = a_2 (a_1 h_0 + b_1) + b_2 the composed form is (a_2 a_1) h_0 + w with
w = fl(a_2 b_1 + b_2), and fl(w) is off by U |w|, where |w| <= |a_2 b_1| + |b_2|
may exceed |h_2| without limit when w and (a_2 a_1) h_0 cancel.  By induction a
partial sum of any grouping is at most m_t = a_t m_{t-1} + |b_t|, m_0 = |h_0|
(each of its terms appears in m_t, with the same factors), so the roundings are
counted against m_t and not against |h_t|; backwards alike, with |dout|.
"""
import numpy as np

U = 2.0 ** -24


def sig(v):
    v = np.asarray(v, np.float64)
    e = np.exp(-np.abs(v))
    return np.where(v >= 0, 1.0 / (1.0 + e), e / (1.0 + e))


def _terms(x, r, i, A, rb, ib, reset, lengths):
    b, L, D = x.shape
    vr, vi = r + (0 if rb is None else rb), i + (0 if ib is None else ib)
    s, gi = sig(vr), sig(vi)
    l = A * s
    with np.errstate(over="ignore", invalid="ignore"):
        a = np.exp(l)
        q = np.maximum(-np.expm1(2 * l), 0.0)
    beta = np.sqrt(q)
    alive = np.ones((b, L), bool)
    if lengths is not None:
        alive = np.arange(L)[None] < np.clip(lengths, 0, L)[:, None]
    rs = np.zeros((b, L), bool) if reset is None else (np.asarray(reset) != 0) & alive
    # relative errors in U
    fin = lambda v: np.where(np.isfinite(v), np.abs(v), 0.0)  # noqa: E731
    es, ei = fin(vr) + 6.0, fin(vi) + 6.0
    el = es + 2.0
    ea = 2.0 + np.abs(l) * el
    eb = 2.0 + 0.5 * np.maximum(el + 6.0, 8.0) + 1.0
    return dict(s=s, gi=gi, l=l, a=a, beta=beta, alive=alive[..., None], rs=rs[..., None], es=es, ei=ei,
                ea=ea, eb=eb)


def forward(x, r, i, A, rb=None, ib=None, reset=None, lengths=None, init=None):
    """dict: h [b,L,D] (zero behind a row's length), fin, and the bounds eh,
    efin of |fp32 - exact| before any rounding of the output."""
    b, L, D = x.shape
    t = _terms(x, r, i, A, rb, ib, reset, lengths)
    xz = np.where(t["alive"], x, 0.0)
    u = t["gi"] * xz
    bt = np.where(t["rs"], u, t["beta"] * u)
    ebt = np.abs(bt) * (t["eb"] + t["ei"] + 2.0) * U
    h = np.zeros((b, D)) if init is None else init.astype(np.float64).copy()
    e = np.zeros((b, D))
    m = np.abs(h)
    H, E, HP, EP = (np.zeros((b, L, D)) for _ in range(4))
    for k in range(L):
        HP[:, k], EP[:, k] = h, e
        with np.errstate(invalid="ignore", over="ignore"):
            n = np.where(t["rs"][:, k], 0.0, t["a"][:, k] * h) + bt[:, k]
            nm = np.where(t["rs"][:, k], 0.0, t["a"][:, k] * m)
            ne = np.where(t["rs"][:, k], 0.0, t["a"][:, k] * e) + nm * (t["ea"][:, k] + 8.0) * U + ebt[:, k]
        nm = nm + np.abs(bt[:, k])
        ne = ne + nm * U
        ok = t["alive"][:, k]
        h, e, m = np.where(ok, n, h), np.where(ok, ne, e), np.where(ok, nm, m)
        H[:, k], E[:, k] = np.where(ok, h, 0.0), np.where(ok, e, 0.0)
    return dict(h=H, fin=h, eh=E, efin=e, hp=HP, ehp=EP, u=u, **t)


def backward(x, r, i, A, rb=None, ib=None, reset=None, lengths=None, init=None, dout=None, dfin=None):
    """Gradients and, under "e" + name, their bounds."""
    f = forward(x, r, i, A, rb, ib, reset, lengths, init)
    b, L, D = x.shape
    a, beta, gi, s, rs, ok = f["a"], f["beta"], f["gi"], f["s"], f["rs"], f["alive"]
    beta = np.where(rs, 1.0, beta)
    do = np.where(ok, dout, 0.0)
    c = np.zeros((b, D)) if dfin is None else dfin.astype(np.float64).copy()
    ec = np.zeros((b, D))
    mc = np.abs(c)
    G, EG = np.zeros((b, L, D)), np.zeros((b, L, D))
    for k in range(L - 1, -1, -1):
        g = do[:, k] + c
        mg = np.abs(do[:, k]) + mc
        eg = ec + mg * U
        live = ok[:, k]
        G[:, k], EG[:, k] = np.where(live, g, 0.0), np.where(live, eg, 0.0)
        nc = np.where(rs[:, k], 0.0, a[:, k] * g)
        nm = np.where(rs[:, k], 0.0, a[:, k] * mg)
        ne = np.where(rs[:, k], 0.0, a[:, k] * eg) + nm * (f["ea"][:, k] + 8.0) * U
        c, ec, mc = np.where(live, nc, c), np.where(live, ne, ec), np.where(live, nm, mc)
    x = np.where(ok, x, 0.0)
    w = beta * gi
    dx = G * w
    edx = EG * w + np.abs(dx) * (f["eb"] + f["ei"] + 3.0) * U
    di = dx * x * (1 - gi)
    edi = edx * np.abs(x) * (1 - gi) + np.abs(di) * (f["ei"] + 6.0) * U
    move = ok & ~rs
    with np.errstate(divide="ignore", invalid="ignore"):
        ub = np.where(move & (beta > 0), a * f["u"] / np.where(beta > 0, beta, 1.0), 0.0)
        hp = np.where(move, f["hp"], 0.0)
        inner = hp - ub
        dl = np.where(move, G * a * inner, 0.0)
        einner = np.where(move, f["ehp"], 0.0) + np.abs(ub) * (f["ea"] + f["eb"] + f["ei"] + 4.0) * U + np.abs(inner) * U
        edl = np.where(move, EG * a * np.abs(inner) + np.abs(G) * a * einner + np.abs(dl) * (f["ea"] + 3.0) * U, 0.0)
    ds = s * (1 - s)
    dr = dl * A * ds
    edr = edl * np.abs(A) * ds + np.abs(dr) * (3 * f["es"] + 4.0) * U
    da = dl * s
    eda = edl * s + np.abs(da) * (f["es"] + 1.0) * U
    # sums: at most 64 successive fp32 additions inside a chunk, then 64 bits
    out = dict(dx=dx, dr=dr, di=di, dinit=c, edx=edx, edr=edr, edi=edi, edinit=ec)
    for name, v, ev in (("dA", da, eda), ("dr_bias", dr, edr), ("di_bias", di, edi)):
        out[name] = v.sum((0, 1))
        out["e" + name] = ev.sum((0, 1)) + 66 * U * np.abs(v).sum((0, 1))
    return out
