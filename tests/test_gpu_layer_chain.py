"""The gated recurrence, the norm with rotation and the SSD scan run together,
as a layer of a hybrid model does: the recurrence's output is the scan's x, the
normed and rotated queries and keys are its C and B.  Forward, gradients back
through all three, and token-by-token decoding from the prefilled states, each
against the 64-bit references chained the same way (fp32 inputs).

Bounds: the scan's own is 1e-4 * (1 + |ref|) element by element, as in the
tests of the scan; what the stages before it lose (1e-6 relative and less) is
small against that.  Going back, an error e in the scan's gradients passes the
linear maps that follow: the recurrence's dx has coefficients >= 0 in dout, so
its own formula applied to the bound bounds it; the norm's dx is at most
rstd * max|w| * sqrt(2) * e * (1 + |n|) (a turn mixes two elements, and the
mean is at most the root mean square)."""
import numpy as np
import pytest
import torch

import glr_ref
import norm_rotate_ref
import oracle
from mamba_ssd_scan_05_amd import ssd

pytestmark = pytest.mark.gpu
DEV = "cuda"
TOL = 1e-4


def layer(b, L, H, P, G, N, seed):
    g = torch.Generator().manual_seed(seed)
    n = lambda *s: torch.randn(s, generator=g)  # noqa: E731
    D = H * P
    t = dict(x=n(b, L, D), r=n(b, L, D), i=n(b, L, D), A=-torch.rand(D, generator=g) - 0.3, rb=n(D), ib=n(D),
             h0=n(b, D), q=2 * n(b, L, G, N), k=2 * n(b, L, G, N), qw=1 + 0.1 * n(N), kw=1 + 0.1 * n(N),
             freqs=10000.0 ** (-torch.arange(N // 2) / (N // 2)), dt=n(b, L, H) - 2, dtb=0.1 * n(H),
             As=-torch.rand(H, generator=g) - 0.5, Ds=n(H), S0=0.1 * n(b, H, P, N))
    t["q"], t["k"] = t["q"] / N ** 0.25, t["k"] / N ** 0.25
    t["qw"], t["kw"] = t["qw"] / N ** 0.25, t["kw"] / N ** 0.25  # scores of order one
    return {k: v.float() for k, v in t.items()}


def forward_ref(t, pos, H, P):
    a = {k: v.double().numpy() for k, v in t.items()}
    f = glr_ref.forward(a["x"], a["r"], a["i"], a["A"], a["rb"], a["ib"], None, None, a["h0"])
    eps = float(np.float32(1e-6))
    C, _ = norm_rotate_ref.forward(a["q"], a["qw"], pos, a["freqs"], eps, False)
    B, _ = norm_rotate_ref.forward(a["k"], a["kw"], pos, a["freqs"], eps, False)
    b, L, D = a["x"].shape
    xs = f["h"].reshape(b, L, H, P)
    y, S = oracle.scan(xs, a["dt"], a["dtb"], a["As"], B, C, a["Ds"], a["S0"])
    return a, f, xs, B, C, y, S, eps


def close(got, ref, what, tol=None):
    got = got.double().cpu().numpy()
    bound = TOL * (1 + np.abs(ref)) if tol is None else tol
    bad = ~(np.abs(got - ref) <= bound)
    assert not bad.any(), "%s: worst %.3g of the bound" % (what, np.nanmax(np.abs(got - ref) / bound))


@pytest.mark.parametrize("b,L,H,P,G,N", [(2, 150, 4, 16, 2, 32), (1, 300, 2, 64, 1, 128)])
def test_forward_and_gradients(b, L, H, P, G, N):
    t = layer(b, L, H, P, G, N, seed=L)
    pos = np.arange(L)[None].repeat(b, 0)
    a, f, xs, B, C, y, S, eps = forward_ref(t, pos, H, P)
    d = {k: v.to(DEV) for k, v in t.items()}
    states = ssd.ssd_glr_states(d["x"])
    h, hf = ssd.ssd_glr_fwd(d["x"], d["r"], d["i"], d["A"], d["rb"], d["ib"], init_state=d["h0"], states=states)
    qo, ko = ssd.ssd_norm_rotate_fwd(d["q"], d["k"], d["qw"], d["kw"], d["freqs"])
    hs = h.view(b, L, H, P)
    out, fin = ssd.ssd_scan_fwd(hs, d["dt"], d["dtb"], d["As"], ko, qo, d["Ds"], d["S0"])
    close(h, f["h"], "recurrence")
    close(out, y, "y")
    close(fin, S, "state")
    g = torch.Generator().manual_seed(7)
    dy, dS = torch.randn((b, L, H, P), generator=g), torch.randn((b, H, P, N), generator=g)
    gs = ssd.ssd_scan_bwd(hs, d["dt"], d["dtb"], d["As"], ko, qo, d["Ds"], d["S0"], dy.to(DEV), dS.to(DEV))
    gn = ssd.ssd_norm_rotate_bwd(d["q"], d["k"], d["qw"], d["kw"], d["freqs"], None, gs["dC"], gs["dB"])
    gr = ssd.ssd_glr_bwd(d["x"], d["r"], d["i"], d["A"], d["rb"], d["ib"], init_state=d["h0"], states=states,
                         dout=gs["dx"].view(b, L, H * P))
    rs = oracle.scan_bwd(xs, a["dt"], a["dtb"], a["As"], B, C, a["Ds"], a["S0"], dy.double().numpy(), dS.double().numpy())
    for k in ("dx", "dB", "dC", "ddt"):
        close(gs[k], rs[k], k)
    for x, w, dn, dref in ((a["q"], a["qw"], "dq", rs["dC"]), (a["k"], a["kw"], "dk", rs["dB"])):
        ref = norm_rotate_ref.backward(x, w, pos, a["freqs"], eps, False, dref, 200)
        rstd = 1 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
        e = (TOL * (1 + np.abs(dref))).max(-1, keepdims=True)
        close(gn[dn], ref["dx"], dn, rstd * np.abs(w).max() * np.sqrt(2) * e * (1 + np.abs(x * rstd)) + ref["edx"])
    dref = rs["dx"].reshape(b, L, H * P)
    args = (a["x"], a["r"], a["i"], a["A"], a["rb"], a["ib"], None, None, a["h0"])
    ref = glr_ref.backward(*args, dout=dref, dfin=None)
    slack = glr_ref.backward(*args, dout=TOL * (1 + np.abs(dref)), dfin=None)
    close(gr["dx"], ref["dx"], "dx", slack["dx"] + ref["edx"])
    close(gr["dinit"], ref["dinit"], "dinit", slack["dinit"] + ref["edinit"])
    close(gr["di"], ref["di"], "di", np.abs(slack["di"]) + ref["edi"])


def test_prefill_then_decode():
    b, L, H, P, G, N, K = 3, 70, 4, 16, 2, 32, 20
    t = layer(b, L + K, H, P, G, N, seed=3)
    start = np.array([0, 1000, 200000])  # each request at its own position
    pos = start[:, None] + np.arange(L + K)
    a, f, xs, B, C, y, S, eps = forward_ref(t, pos, H, P)
    d = {k: v.to(DEV) for k, v in t.items()}
    p = torch.tensor(pos, device=DEV)
    cut = lambda k: d[k][:, :L].contiguous()  # noqa: E731
    h, hf = ssd.ssd_glr_fwd(cut("x"), cut("r"), cut("i"), d["A"], d["rb"], d["ib"], init_state=d["h0"])
    qo, ko = ssd.ssd_norm_rotate_fwd(d["q"][:, :L], d["k"][:, :L], d["qw"], d["kw"], d["freqs"], p[:, :L].contiguous())
    out, Sg = ssd.ssd_scan_fwd(h.view(b, L, H, P), cut("dt"), d["dtb"], d["As"], ko, qo, d["Ds"], d["S0"])
    close(out, y[:, :L], "prefill")
    for k in range(L, L + K):
        hk = ssd.ssd_glr_step(hf, d["x"][:, k], d["r"][:, k], d["i"][:, k], d["A"], d["rb"], d["ib"])
        qk, kk = ssd.ssd_norm_rotate_fwd(d["q"][:, k:k + 1], d["k"][:, k:k + 1], d["qw"], d["kw"], d["freqs"],
                                         p[:, k:k + 1].contiguous())
        delta = torch.nn.functional.softplus(d["dt"][:, k] + d["dtb"])
        yk = ssd.ssd_step(Sg, hk.view(b, H, P), delta, d["As"], kk[:, 0].contiguous(), qk[:, 0].contiguous(), d["Ds"])
        close(yk, y[:, k], "token %d" % k)
    close(hf, f["fin"], "recurrent state")
    close(Sg, S, "scan state")


def within(got, ref, bound, what):
    """Within the reference's bound and half a step of got's type."""
    half = torch.finfo(got.dtype).eps / 2
    got = got.double().cpu().numpy()
    tol = bound + half * (np.abs(ref) + bound) + 1e-37
    assert np.all(np.abs(got - ref) <= tol), "%s: worst %.3g of the bound" % (what, np.max(np.abs(got - ref) / tol))


@pytest.mark.parametrize("b,L,H,P,G,N", [(2, 150, 4, 16, 2, 32), (1, 300, 2, 64, 1, 128)])
def test_bf16_training(b, L, H, P, G, N):
    # bf16 activations through all three and back, without a cast: the scan's
    # fp32 gradients go into the other two as they are.  Each stage against its
    # reference on what it was given; the scan's bound for bf16 is
    # 2e-2 * (1 + |ref|), as in its own tests.
    bf = torch.bfloat16
    t = layer(b, L, H, P, G, N, seed=L + 1)
    d = {k: v.to(DEV).to(bf) if k in ("x", "r", "i", "q", "k") else v.to(DEV) for k, v in t.items()}
    a = {k: v.double().cpu().numpy() for k, v in d.items()}
    pos, eps = np.arange(L)[None].repeat(b, 0), float(np.float32(1e-6))
    gates = (d["x"], d["r"], d["i"], d["A"], d["rb"], d["ib"])
    ref_gates = tuple(a[k] for k in ("x", "r", "i", "A", "rb", "ib")) + (None, None, a["h0"])
    states = ssd.ssd_glr_states(d["x"])
    h, hf = ssd.ssd_glr_fwd(*gates, init_state=d["h0"], states=states)
    C, B = ssd.ssd_norm_rotate_fwd(d["q"], d["k"], d["qw"], d["kw"], d["freqs"])
    hs = h.view(b, L, H, P)
    scan = (d["dt"], d["dtb"], d["As"], B, C, d["Ds"], d["S0"])
    out, fin = ssd.ssd_scan_fwd(hs, *scan)
    f = glr_ref.forward(*ref_gates)
    within(h, f["h"], f["eh"], "h")
    for y, x, w in ((C, "q", "qw"), (B, "k", "kw")):
        within(y, *norm_rotate_ref.forward(a[x], a[w], pos, a["freqs"], eps, False), x)
    num = lambda v: v.double().cpu().numpy()  # noqa: E731
    ref_scan = (num(hs), a["dt"], a["dtb"], a["As"], num(B), num(C), a["Ds"], a["S0"])
    y, S = oracle.scan(*ref_scan)
    close(out, y, "y", 2e-2 * (1 + np.abs(y)))
    close(fin, S, "state", 2e-2 * (1 + np.abs(S)))
    g = torch.Generator().manual_seed(8)
    dy, dS = torch.randn((b, L, H, P), generator=g).to(bf), torch.randn((b, H, P, N), generator=g)
    gs = ssd.ssd_scan_bwd(hs, *scan, dy.to(DEV), dS.to(DEV))
    rs = oracle.scan_bwd(*ref_scan, dy.double().numpy(), dS.double().numpy())
    for k in ("dx", "dB", "dC"):
        close(gs[k], rs[k], k, 2e-2 * (1 + np.abs(rs[k])))
    gn = ssd.ssd_norm_rotate_bwd(d["q"], d["k"], d["qw"], d["kw"], d["freqs"], None, gs["dC"], gs["dB"])
    gr = ssd.ssd_glr_bwd(*gates, init_state=d["h0"], states=states, dout=gs["dx"].view(b, L, H * P))
    for x, w, dn, wn, dy in (("q", "qw", "dq", "dq_weight", gs["dC"]), ("k", "kw", "dk", "dk_weight", gs["dB"])):
        ref = norm_rotate_ref.backward(a[x], a[w], pos, a["freqs"], eps, False, num(dy), 200)
        assert gn[dn].dtype == bf
        within(gn[dn], ref["dx"], ref["edx"], dn)
        within(gn[wn], ref["dw"], ref["edw"], wn)
    ref = glr_ref.backward(*ref_gates, dout=num(gs["dx"]).reshape(b, L, H * P), dfin=None)
    for k in ("dx", "dr", "di", "dA", "dr_bias", "di_bias", "dinit"):
        assert gr[k].dtype == (bf if k in ("dx", "dr", "di") else torch.float32)
        within(gr[k], ref[k], ref["e" + k], k)
