"""Norm and rotation of queries and keys on the GPU against the 64-bit
reference: every element within the reference's rounding bound plus half a
step of the output's type."""
import sys

import numpy as np
import pytest
import torch

import norm_rotate_ref as ref
from mamba_ssd_scan_05_amd import ssd

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF, F32 = torch.bfloat16, torch.float32


def say(*a):
    print(*a, file=sys.stderr, flush=True)


def make(b, L, Hq, Hk, N, npair, dtype, layout="dense", far=0, i64=False, explicit=True, weights=True, seed=1):
    g = torch.Generator().manual_seed(seed)
    n = lambda *s: torch.randn(s, generator=g)  # noqa: E731
    if layout == "fused":
        proj = (3 * n(b, L, Hq + 2 * Hk, N)).to(dtype).to(DEV)
        q, k = proj[:, :, :Hq], proj[:, :, Hq:Hq + Hk]
    elif layout == "offset":  # heads that start between 4-element boundaries
        proj = n(b, L, (Hq + Hk) * N + 7).to(dtype).to(DEV)
        q, k = proj[..., 3:3 + Hq * N].unflatten(-1, (Hq, N)), proj[..., 5 + Hq * N:5 + (Hq + Hk) * N].unflatten(-1, (Hk, N))
    elif layout == "heads_first":
        q, k = (n(b, H, L, N).to(dtype).to(DEV).transpose(1, 2) for H in (Hq, Hk))
    elif layout == "shared":  # one key head spread over all
        q, k = n(b, L, Hq, N).to(dtype).to(DEV), n(b, L, 1, N).to(dtype).to(DEV).expand(b, L, Hk, N)
    else:
        q, k = (n(b, L, H, N).to(dtype).to(DEV) for H in (Hq, Hk))
    pos = (torch.randint(-far, far + 1, (b, L), generator=g) if far else
           torch.arange(L).expand(b, L).contiguous())
    t = dict(q=q, k=k, q_weight=n(N).to(DEV) if weights else None, k_weight=n(N).to(DEV) if weights else None,
             freqs=(10000.0 ** (-torch.arange(npair, dtype=torch.float64) / max(npair, 1))).float().to(DEV) if npair else None,
             positions=pos.to(torch.int64 if i64 else torch.int32).to(DEV) if explicit else None)
    return t, pos.numpy(), n(b, L, Hq, N).to(dtype).to(DEV), n(b, L, Hk, N).to(dtype).to(DEV)


def num(t):
    return None if t is None else t.float().cpu().double().numpy()


def check(name, got, want, bound):
    half = torch.finfo(got.dtype).eps / 2
    got = got.float().cpu().double().numpy()
    tol = bound + half * (np.abs(want) + bound) + 1e-37
    bad = ~(np.abs(got - want) <= tol)
    assert not bad.any(), "%s: %d of %d beyond the bound, worst %.3g of it at %s" % (
        name, bad.sum(), bad.size, np.nanmax(np.abs(got - want) / tol), np.argwhere(bad)[0])


CASES = [
    # b, L, Hq, Hk, N, npair, layout, far, i64
    (1, 1, 1, 1, 8, 4, "dense", 0, False),
    (1, 1, 1, 1, 16, 8, "dense", 5000, True),
    (2, 3, 5, 1, 24, 4, "dense", 0, False),
    (3, 17, 3, 2, 32, 16, "fused", 100000, False),
    (1, 65, 2, 1, 40, 0, "dense", 0, False),
    (2, 33, 7, 7, 64, 32, "heads_first", 1 << 20, False),
    (1, 9, 6, 2, 80, 20, "offset", 4096, True),
    (2, 31, 4, 4, 96, 48, "shared", 0, False),
    (32, 1, 32, 8, 128, 64, "fused", 131072, False),
    (1, 300, 1, 1, 128, 64, "dense", 0, False),
    (1, 11, 9, 3, 192, 32, "fused", 1 << 30, True),
    (2, 13, 2, 1, 256, 128, "dense", 1 << 21, False),
    (1, 5000, 2, 1, 16, 8, "dense", 0, False),
]


@pytest.mark.parametrize("dtype", [F32, BF], ids=["f32", "bf16"])
@pytest.mark.parametrize("interleaved", [False, True], ids=["halves", "adjacent"])
@pytest.mark.parametrize("case", CASES, ids=["b%d_L%d_Hq%d_Hk%d_N%d_p%d_%s" % c[:7] for c in CASES])
def test_forward_and_gradients(case, interleaved, dtype):
    b, L, Hq, Hk, N, npair, layout, far, i64 = case
    say("norm_rotate", case, interleaved, dtype)
    t, pos, dyq, dyk = make(b, L, Hq, Hk, N, npair, dtype, layout, far, i64, explicit=far > 0 or i64, weights=N != 24)
    f = num(t["freqs"])
    qo, ko = ssd.ssd_norm_rotate_fwd(**t, eps=1e-5, interleaved=interleaved)
    g = ssd.ssd_norm_rotate_bwd(**t, dq_out=dyq, dk_out=dyk, eps=1e-5, interleaved=interleaved)
    torch.cuda.synchronize()
    eps = float(np.float32(1e-5))
    for x, w, o, dy, dn, wn in ((t["q"], t["q_weight"], qo, dyq, "dq", "dq_weight"),
                                (t["k"], t["k_weight"], ko, dyk, "dk", "dk_weight")):
        y, ey = ref.forward(num(x), num(w), pos, f, eps, interleaved)
        check("y", o, y, ey)
        rows = b * L * (Hq + Hk)
        d = ref.backward(num(x), num(w), pos, f, eps, interleaved, num(dy), 130 + Hq + Hk + rows // 1024)
        check(dn, g[dn], d["dx"], d["edx"])
        check(wn, g[wn], d["dw"], d["edw"])


def test_views_of_the_gradients_and_no_weight_gradients():
    t, pos, dyq, dyk = make(2, 40, 4, 2, 64, 32, BF)
    want = ssd.ssd_norm_rotate_bwd(**t, dq_out=dyq, dk_out=dyk)
    both = torch.cat([dyq, dyk], 2)
    g = ssd.ssd_norm_rotate_bwd(**t, dq_out=both[:, :, :4], dk_out=both[:, :, 4:], want_weights=False)
    assert g["dq_weight"] is None and torch.equal(g["dq"], want["dq"]) and torch.equal(g["dk"], want["dk"])
    # a gradient that is one row for every token (what a mean's backward gives)
    row = torch.randn(1, 1, 4, 64, device=DEV).to(BF)
    a = ssd.ssd_norm_rotate_bwd(**t, dq_out=row.expand(2, 40, 4, 64), dk_out=dyk)
    c = ssd.ssd_norm_rotate_bwd(**t, dq_out=row.expand(2, 40, 4, 64).contiguous(), dk_out=dyk)
    for n in a:
        assert torch.equal(a[n], c[n]), n


def test_zero_vectors_and_negative_positions():
    t, pos, dyq, dyk = make(1, 6, 2, 2, 32, 16, F32, far=1000)
    t["q"][:, 2] = 0
    qo, ko = ssd.ssd_norm_rotate_fwd(**t, eps=1e-6)
    g = ssd.ssd_norm_rotate_bwd(**t, dq_out=dyq, dk_out=dyk, eps=1e-6)
    assert bool((qo[:, 2] == 0).all()) and bool(torch.isfinite(g["dq"]).all())
    # turning there and back again is the normed vector
    back = dict(t, positions=-t["positions"])
    one = dict(q_weight=None, k_weight=None, freqs=back["freqs"], positions=back["positions"])
    n, _ = ssd.ssd_norm_rotate_fwd(t["q"], t["k"], t["q_weight"], t["k_weight"], None, None, eps=1e-6)
    q2, _ = ssd.ssd_norm_rotate_fwd(qo, ko, **one, eps=0.0)
    rms = n.pow(2).mean(-1, keepdim=True).sqrt()
    live = rms[..., 0] > 0
    # two passes of 23 U (|u| + |v|) each and the two norms
    assert float(((q2 - n / rms)[live]).abs().max()) <= 80 * ref.U * float((n / rms)[live].abs().max())


def test_gradients_against_differences():
    t, pos, dyq, dyk = make(2, 7, 3, 1, 32, 8, F32, far=300)
    g = ssd.ssd_norm_rotate_bwd(**t, dq_out=dyq, dk_out=dyk)
    rng = np.random.default_rng(3)
    eps = float(np.float32(1e-6))
    for x, w, dy, dn, wn in ((t["q"], t["q_weight"], dyq, "dq", "dq_weight"), (t["k"], t["k_weight"], dyk, "dk", "dk_weight")):
        x, w, dy = num(x), num(w), num(dy)
        vx, vw, h = rng.standard_normal(x.shape), rng.standard_normal(w.shape), 1e-5
        F = lambda x, w: float((ref.forward(x, w, pos, num(t["freqs"]), eps, False)[0] * dy).sum())  # noqa: E731
        d = (F(x + h * vx, w + h * vw) - F(x - h * vx, w - h * vw)) / (2 * h)
        p = [num(g[dn]) * vx, num(g[wn]) * vw]
        assert abs(p[0].sum() + p[1].sum() - d) <= 1e-5 * sum(np.abs(v).sum() for v in p)


def test_repeats_graphs_and_streams():
    t, pos, dyq, dyk = make(4, 500, 8, 2, 128, 64, BF, "fused")
    want = ssd.ssd_norm_rotate_fwd(**t)
    wg = ssd.ssd_norm_rotate_bwd(**t, dq_out=dyq, dk_out=dyk)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        ssd.ssd_norm_rotate_bwd(**t, dq_out=dyq, dk_out=dyk)
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        qo, ko = ssd.ssd_norm_rotate_fwd(**t)
        g = ssd.ssd_norm_rotate_bwd(**t, dq_out=dyq, dk_out=dyk)
    for k in range(4):
        for v in (qo, ko, *g.values()):
            v.fill_(float("nan"))
        graph.replay()
        e = ssd.ssd_norm_rotate_bwd(**t, dq_out=dyq, dk_out=dyk, stream=s.cuda_stream if k % 2 else None)
        torch.cuda.synchronize()
        assert torch.equal(qo, want[0]) and torch.equal(ko, want[1])
        for n in wg:
            assert torch.equal(g[n], wg[n]) and torch.equal(e[n], wg[n]), (k, n)


def test_far_offsets():
    t, pos, _, _ = make(2, 3, 2, 1, 64, 32, BF)
    want = ssd.ssd_norm_rotate_fwd(**t)
    big = torch.empty((1 << 31) + (1 << 16), dtype=BF, device=DEV)
    q = big.as_strided((2, 3, 2, 64), (1 << 31, 128, 64, 1))
    q.copy_(t["q"])
    got = ssd.ssd_norm_rotate_fwd(**dict(t, q=q))
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    # heads 2^30 elements apart, as in a heads-first cache of long sequences
    q = big.as_strided((2, 3, 2, 64), (192, 64, 1 << 30, 1))
    q.copy_(t["q"])
    dy = [torch.randn_like(v) for v in want]
    got = ssd.ssd_norm_rotate_fwd(**dict(t, q=q))
    wg = ssd.ssd_norm_rotate_bwd(**t, dq_out=dy[0], dk_out=dy[1])
    g = ssd.ssd_norm_rotate_bwd(**dict(t, q=q), dq_out=dy[0], dk_out=dy[1])
    assert torch.equal(got[0], want[0]) and all(torch.equal(g[k], wg[k]) for k in wg)


def test_one_weight_and_shared_inputs():
    t, pos, dyq, dyk = make(2, 9, 3, 3, 40, 8, F32)
    t["q_weight"] = None
    t["k"] = t["q"]
    qo, ko = ssd.ssd_norm_rotate_fwd(**t)
    g = ssd.ssd_norm_rotate_bwd(**t, dq_out=dyq, dk_out=dyk, out=dict(dk_weight=torch.empty(40, device=DEV)))
    eps = float(np.float32(1e-6))
    for w, o, dy, dn, wn in ((None, qo, dyq, "dq", "dq_weight"), (t["k_weight"], ko, dyk, "dk", "dk_weight")):
        y, ey = ref.forward(num(t["q"]), num(w), pos, num(t["freqs"]), eps, False)
        check("y", o, y, ey)
        d = ref.backward(num(t["q"]), num(w), pos, num(t["freqs"]), eps, False, num(dy), 140)
        check(dn, g[dn], d["dx"], d["edx"])
        check(wn, g[wn], d["dw"], d["edw"])


def test_many_tokens_of_few_heads_and_few_tokens_of_many():
    for b, L, Hq, Hk, N, npair in ((1, 200000, 1, 1, 16, 8), (1, 2, 300, 77, 32, 16), (3, 1, 1, 1, 256, 64)):
        t, pos, dyq, dyk = make(b, L, Hq, Hk, N, npair, F32)
        qo, ko = ssd.ssd_norm_rotate_fwd(**t)
        g = ssd.ssd_norm_rotate_bwd(**t, dq_out=dyq, dk_out=dyk)
        eps = float(np.float32(1e-6))
        for x, w, o, dy, dn, wn in ((t["q"], t["q_weight"], qo, dyq, "dq", "dq_weight"),
                                    (t["k"], t["k_weight"], ko, dyk, "dk", "dk_weight")):
            y, ey = ref.forward(num(x), num(w), pos, num(t["freqs"]), eps, False)
            check("y", o, y, ey)
            d = ref.backward(num(x), num(w), pos, num(t["freqs"]), eps, False, num(dy), 130 + Hq + Hk + b * L * (Hq + Hk) // 1024)
            check(dn, g[dn], d["dx"], d["edx"])
            check(wn, g[wn], d["dw"], d["edw"])


def inverse_turn():
    """1 / (2 pi) to 60 digits."""
    from fractions import Fraction as Q

    def arctan_of_inverse(n):
        total, term, k = Q(0), Q(1, n), 1
        while abs(term) > Q(1, 10 ** 62):
            total, term, k = total + term / k, -term / (n * n), k + 2
        return total

    return 1 / (8 * (4 * arctan_of_inverse(5) - arctan_of_inverse(239)))


@pytest.mark.parametrize("i64", [False, True], ids=["i32", "i64"])
def test_far_positions_against_exact_turns(i64):
    # angles reduced with rational arithmetic: the fraction of a turn is exact
    # here, its angle good to 2^-52
    from fractions import Fraction as Q
    pos = [0, 1, 105413503, (1 << 24) - 1, (1 << 27) + 1, (1 << 30) - 1, (1 << 31) - 1, -(1 << 31)]
    if i64:
        pos += [(1 << 36) + 12345, (1 << 40) - 7, -(1 << 45) - 1, (1 << 50) + 3, (1 << 52) + 1, (1 << 53) - 1, 1 << 53,
                -(1 << 53)]
    L, N = len(pos), 32
    freqs = torch.tensor([1.0, 0.75, 0.1, 10000.0 ** -0.25, 1e-4, 3.1415927, 100.0, 2.0 ** -30], dtype=torch.float32)
    t, _, _, _ = make(1, L, 2, 1, N, 8, F32, weights=False, explicit=False)
    t.update(freqs=freqs.to(DEV), positions=torch.tensor([pos], dtype=torch.int64 if i64 else torch.int32, device=DEV))
    turn = inverse_turn()
    ang = np.array([[float((p * Q(float(f)) * turn) % 1) * 2 * np.pi for f in freqs] for p in pos])
    c, s = np.cos(ang)[None, :, None], np.sin(ang)[None, :, None]
    eps = float(np.float32(1e-6))
    for inter in (False, True):
        qo, ko = ssd.ssd_norm_rotate_fwd(**t, interleaved=inter)
        for x, o in ((t["q"], qo), (t["k"], ko)):
            x = num(x)
            u = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
            a, b = (u[..., 0:16:2], u[..., 1:16:2]) if inter else (u[..., :8], u[..., 8:16])
            y = u.copy()
            if inter:
                y[..., 0:16:2], y[..., 1:16:2] = a * c - b * s, a * s + b * c
            else:
                y[..., :8], y[..., 8:16] = a * c - b * s, a * s + b * c
            both = np.abs(u)
            tot = np.abs(a) + np.abs(b)
            if inter:
                both[..., 0:16:2] = both[..., 1:16:2] = tot
            else:
                both[..., :8] = both[..., 8:16] = tot
            check("y", o, y, 23 * ref.U * both)  # the bound of norm_rotate_ref.forward


@pytest.mark.parametrize("dtype", [F32, BF], ids=["f32", "bf16"])
@pytest.mark.parametrize("N,npair", [(8, 4), (40, 8), (128, 64), (256, 0)])
def test_mean_squares_outside_the_range_of_fp32(N, npair, dtype):
    # heads of very small and very large elements beside ordinary ones, no eps
    t, pos, dyq, dyk = make(2, 6, 3, 1, N, npair, dtype, seed=5)
    scale = torch.tensor([1e-36, 1e-30, 1e-22, 1.0, 1e18, 1e30], device=DEV).view(1, 6, 1, 1)
    t["q"], t["k"] = (t["q"].float() * scale).to(dtype), (t["k"].float() * scale.flip(1)).to(dtype)
    t["q"][0, 3, 1, N // 2] = 1e-25  # one tiny element in an ordinary head
    qo, ko = ssd.ssd_norm_rotate_fwd(**t, eps=0.0)
    g = ssd.ssd_norm_rotate_bwd(**t, dq_out=dyq, dk_out=dyk, eps=0.0)
    for x, w, o, dy, dn, wn in ((t["q"], t["q_weight"], qo, dyq, "dq", "dq_weight"),
                                (t["k"], t["k_weight"], ko, dyk, "dk", "dk_weight")):
        y, ey = ref.forward(num(x), num(w), pos, num(t["freqs"]), 0.0, False)
        check("y", o, y, ey)
        d = ref.backward(num(x), num(w), pos, num(t["freqs"]), 0.0, False, num(dy), 140)
        # gradients below 2^-126 count as 0
        check(dn, g[dn], d["dx"], d["edx"] + 2.0 ** -126)
        check(wn, g[wn], d["dw"], d["edw"])
    # the largest element of the contract, with an ordinary eps: 256 squares of
    # 2^59 sum to 2^126
    t["q"] = torch.full_like(t["q"], 2.0 ** 59)
    qo, _ = ssd.ssd_norm_rotate_fwd(t["q"], t["k"], eps=1e-6)
    assert float((qo.float() - 1).abs().max()) <= 13 * ref.U + torch.finfo(dtype).eps / 2


def test_weight_gradients_of_very_many_tokens():
    # one head vector for all of 2^23 tokens (stride 0): 2048 of them to every
    # wave.  The sums of equal terms are exact but for fp32's roundings, which
    # may number a few dozen at each level however many tokens there are (64
    # items in registers, 32 such sums, 8 lane groups).
    L, N = 1 << 23, 256
    t, _, dyq, dyk = make(1, 1, 1, 1, N, 0, BF, seed=6)
    g = ssd.ssd_norm_rotate_bwd(t["q"].expand(1, L, 1, N), t["k"].expand(1, L, 1, N), t["q_weight"], t["k_weight"], None,
                                None, dyq.expand(1, L, 1, N), dyk.expand(1, L, 1, N))
    for x, w, dy, dn, wn in ((t["q"], t["q_weight"], dyq, "dq", "dq_weight"), (t["k"], t["k_weight"], dyk, "dk", "dk_weight")):
        d = ref.backward(num(x), num(w), np.zeros((1, 1)), None, float(np.float32(1e-6)), False, num(dy), 64 + 32 + 8)
        check(wn, g[wn], L * d["dw"], L * d["edw"])
        check(dn, g[dn][:, -1:], d["dx"], d["edx"])
        assert bool((g[dn] == g[dn][:, :1]).all())


@pytest.mark.parametrize("interleaved", [False, True], ids=["halves", "adjacent"])
@pytest.mark.parametrize("case", CASES, ids=["b%d_L%d_Hq%d_Hk%d_N%d_p%d_%s" % c[:7] for c in CASES])
def test_gradients_from_fp32_output_gradients(case, interleaved):
    b, L, Hq, Hk, N, npair, layout, far, i64 = case
    t, pos, _, _ = make(b, L, Hq, Hk, N, npair, BF, layout, far, i64, explicit=far > 0 or i64)
    g = torch.Generator().manual_seed(7)
    pad = 1 if layout == "offset" else 0  # rows between 16-byte boundaries
    dyq, dyk = (torch.randn(b, L, H, N + pad, generator=g).to(DEV)[..., pad:] for H in (Hq, Hk))
    got = ssd.ssd_norm_rotate_bwd(**t, dq_out=dyq, dk_out=dyk, eps=1e-5, interleaved=interleaved)
    rows = b * L * (Hq + Hk)
    for x, w, dy, dn, wn in ((t["q"], t["q_weight"], dyq, "dq", "dq_weight"), (t["k"], t["k_weight"], dyk, "dk", "dk_weight")):
        assert got[dn].dtype == BF
        d = ref.backward(num(x), num(w), pos, num(t["freqs"]), float(np.float32(1e-5)), interleaved, num(dy),
                         130 + Hq + Hk + rows // 1024)
        check(dn, got[dn], d["dx"], d["edx"])
        check(wn, got[wn], d["dw"], d["edw"])


def test_one_weight_gradient_or_none():
    t, pos, dyq, dyk = make(2, 300, 4, 2, 64, 32, BF)
    want = ssd.ssd_norm_rotate_bwd(**t, dq_out=dyq, dk_out=dyk)
    ws = torch.empty(ssd.ssd_norm_rotate_workspace(64), dtype=torch.uint8, device=DEV)
    for which in ((), ("dq_weight",), ("dk_weight",)):
        out = {k: torch.empty_like(want[k]) if k in which or k in ("dq", "dk") else None for k in ("dq", "dk", "dq_weight", "dk_weight")}
        keep, d = ssd._descs(*t.values(), dyq, dyk, *out.values())
        st = ssd.lib().ssd_norm_rotate_bwd(*d, 1e-6, 0, ws.data_ptr() if which else None, ws.numel() if which else 0,
                                           torch.cuda.current_stream().cuda_stream)
        assert st == 0, ssd.ssd_last_error()
        for k, v in out.items():
            assert v is None or torch.equal(v, want[k]), (which, k)
