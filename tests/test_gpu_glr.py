"""Gated linear recurrence on the GPU against the 64-bit reference: every
output element within the reference's rounding bound plus half a step of the
output's type."""
import sys

import numpy as np
import pytest
import torch

import glr_ref
from mamba_ssd_scan_05_amd import ssd

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF, F32 = torch.bfloat16, torch.float32


def say(*a):
    print(*a, file=sys.stderr, flush=True)


def make(b, L, D, dtype, seed, layout="dense", reset=0.0, lengths=None, init=True, bias=True, amin=0.001, amax=0.7):
    g = torch.Generator().manual_seed(seed)
    n = lambda *s: torch.randn(s, generator=g)  # noqa: E731
    if layout == "fused":
        proj = n(b, L, 3 * D).to(dtype).to(DEV)
        x, r, i = proj[..., :D], proj[..., D:2 * D], proj[..., 2 * D:]
    elif layout == "offset":  # rows that start between 16-byte boundaries
        proj = n(b, L, 3 * D + 5).to(dtype).to(DEV)
        x, r, i = proj[..., 1:D + 1], proj[..., D + 2:2 * D + 2], proj[..., 2 * D + 3:3 * D + 3]
    elif layout == "time_major":
        x, r, i = (n(L, b, D).to(dtype).to(DEV).transpose(0, 1) for _ in range(3))
    elif layout == "broadcast":  # one row of gates for the whole batch
        x = n(b, L, D).to(dtype).to(DEV)
        r, i = n(1, L, D).to(dtype).to(DEV).expand(b, L, D), n(b, 1, D).to(dtype).to(DEV).expand(b, L, D)
    else:
        x, r, i = (n(b, L, D).to(dtype).to(DEV) for _ in range(3))
    # decays spread over the scale of their logarithm
    A = -torch.exp(torch.empty(D).uniform_(np.log(amin), np.log(amax), generator=g)).to(DEV)
    t = dict(x=x, r=r, i=i, A=A, r_bias=n(D).to(DEV) if bias else None, i_bias=n(D).to(DEV) if bias else None,
             reset=(torch.rand(b, L, generator=g) < reset).to(torch.uint8).to(DEV) if reset else None,
             lengths=None if lengths is None else torch.tensor(lengths, dtype=torch.int32, device=DEV),
             init_state=n(b, D).to(DEV) if init else None)
    return t, n(b, L, D).to(dtype).to(DEV), n(b, D).to(DEV)


def host(t):
    names = dict(r_bias="rb", i_bias="ib", init_state="init")
    return {names.get(k, k): None if v is None else
            (v.cpu().numpy() if v.dtype in (torch.uint8, torch.int32) else v.float().cpu().double().numpy())
            for k, v in t.items()}


def check(name, got, want, bound):
    half = torch.finfo(got.dtype).eps / 2
    got = got.float().cpu().double().numpy()
    tol = bound + half * (np.abs(want) + bound) + 1e-37
    bad = ~(np.abs(got - want) <= tol)
    assert not bad.any(), "%s: %d of %d beyond the bound, worst %.3g of it at %s" % (
        name, bad.sum(), bad.size, np.nanmax(np.abs(got - want) / tol), np.argwhere(bad)[0])


SHAPES = [
    # b, L, D, layout, reset, lengths, init
    (1, 1, 1, "dense", 0, None, True),
    (1, 1, 64, "dense", 0, None, False),
    (2, 2, 72, "fused", 0.5, [0, 2], True),
    (3, 5, 3, "dense", 0, None, True),
    (3, 16, 200, "dense", 0.05, [16, 9, 1], True),
    (2, 33, 130, "fused", 0, None, True),
    (2, 64, 128, "fused", 0.02, [64, 33], False),
    (3, 65, 40, "offset", 0, None, True),
    (2, 127, 40, "dense", 0.02, None, True),
    (1, 128, 130, "dense", 0, None, True),
    (2, 129, 64, "offset", 0.01, [129, 128], True),
    (3, 130, 128, "fused", 0.02, [65, 64, 63], True),
    (2, 200, 256, "dense", 0, [16, 17], True),
    (1, 255, 56, "fused", 0, None, False),
    (5, 150, 66, "time_major", 0.01, [150, 0, 149, 64, 150], True),
    (2, 256, 8, "dense", 0, None, True),
    (4, 257, 96, "broadcast", 0.01, [257, 256, 1, 0], True),
    (3, 513, 33, "fused", 0.004, [511, 513, 257], True),
    (2, 1000, 72, "dense", 0, None, True),
    (1, 3000, 65, "dense", 0, None, False),      # more chunks than one look back covers
    (3, 2311, 136, "fused", 0.0008, [2311, 100, 1300], True),
    (1, 700, 64, "dense", 1.0, None, True),      # every token starts a document
]


@pytest.mark.parametrize("dtype", [F32, BF], ids=["f32", "bf16"])
@pytest.mark.parametrize("case", SHAPES, ids=["b%d_L%d_D%d_%s" % c[:4] for c in SHAPES])
def test_forward_and_gradients(case, dtype):
    b, L, D, layout, reset, lengths, init = case
    say("glr", case, dtype)
    t, dout, dfin = make(b, L, D, dtype, seed=L + D, layout=layout, reset=reset, lengths=lengths, init=init,
                         bias=L % 2 == 1)
    h = host(t)
    f = glr_ref.forward(**h)
    states = ssd.ssd_glr_states(t["x"]).fill_(float("nan"))
    out = torch.full((b, L, D), 7.0, dtype=dtype, device=DEV)
    fin = torch.full((b, D), float("nan"), device=DEV)
    ssd.ssd_glr_fwd(**t, out=out, final_state=fin, states=states)
    torch.cuda.synchronize()
    alive = f["alive"]
    assert bool((out.float().cpu().numpy()[~np.broadcast_to(alive, out.shape)] == 7.0).all()), "wrote behind a row"
    check("out", torch.where(torch.tensor(alive, device=DEV), out, 0), f["h"], f["eh"])
    check("final", fin, f["fin"], f["efin"])
    st = states.cpu().double().numpy()
    for s in range(states.shape[1]):
        for row in range(b):
            n = L if lengths is None else lengths[row]
            k = s * ssd.SSD_GLR_SEGMENT
            if s == 0 or k < n:
                assert np.all(np.abs(st[row, s] - f["hp"][row, k]) <=
                              f["ehp"][row, k] + glr_ref.U * np.abs(f["hp"][row, k])), (row, s)
    ref = glr_ref.backward(**h, dout=dout.float().cpu().double().numpy(), dfin=dfin.cpu().double().numpy())
    for saved in (states, None):
        pre = {k: torch.full((b, L, D), float("nan"), dtype=dtype, device=DEV) for k in ("dx", "dr", "di")}
        g = ssd.ssd_glr_bwd(**t, dout=dout, dfinal_state=dfin, states=saved, out=pre)
        torch.cuda.synchronize()
        for k in ("dx", "dr", "di", "dA", "dr_bias", "di_bias", "dinit"):
            check(k, g[k], ref[k], ref["e" + k])


def test_extreme_gates():
    # gates fully open and shut, decays of zero, none and above one, channels
    # whose factor sqrt(1 - a^2) is exactly 0
    b, L, D = 2, 300, 24
    t, dout, dfin = make(b, L, D, F32, seed=3)
    t["A"][:8] = torch.tensor([0.0, -1e-30, -1e-7, -1e-4, -50.0, -1000.0, -0.0, 1e-3], device=DEV)
    t["r"][:, ::7] = 90.0
    t["r"][:, 1::7] = -90.0
    t["r"][0, 2::7] = float("inf")
    t["i"][:, ::5] = -120.0
    t["i"][:, 1::5] = 120.0
    h = host(t)
    f = glr_ref.forward(**h)
    out, fin = ssd.ssd_glr_fwd(**t)
    # fp32 denormals count as 0: a gate s below 2^-126 does, which moves 1 - a^2
    # by at most 2 |A| 2^-126 and its root by sqrt(2000 * 2^-126) < 4.9e-18 for
    # |A| <= 1000, once a token, times |u| <= max |x|; a decay passes on no more
    # than it receives, except channel 7 (A = 1e-3, factor 0, not affected)
    slack = 4.9e-18 * L * float(t["x"].abs().max())
    check("out", out, f["h"], f["eh"] + slack)
    check("final", fin, f["fin"], f["efin"] + slack)
    g = ssd.ssd_glr_bwd(**t, dout=dout, dfinal_state=dfin)
    for k in ("dx", "dr", "di", "dA", "dr_bias", "di_bias", "dinit"):
        assert bool(torch.isfinite(g[k]).all()), k
    ref = glr_ref.backward(**h, dout=dout.cpu().double().numpy(), dfin=dfin.cpu().double().numpy())
    keep = np.ones(D, bool)
    keep[1] = False  # a factor below fp32's normal range: its gradient is that of 0 or of a tiny number
    for k in ("dx", "di", "dinit"):
        # the same flush of the factor, times |g| <= L max(|dout|, |dfinal|)
        # (channel 7: times e^0.3) and |x|
        check(k, g[k][..., torch.tensor(keep, device=DEV)], ref[k][..., keep],
              (ref["e" + k] + slack * 1.5 * float(torch.maximum(dout.abs().max(), dfin.abs().max())))[..., keep])


def test_garbage_does_not_pass_a_reset_or_a_length():
    b, L, D = 3, 700, 40
    nan, inf = float("nan"), float("inf")
    for dtype in (F32, BF):
        t, dout, dfin = make(b, L, D, dtype, seed=4, lengths=[300, 700, 0])
        t["reset"] = torch.zeros(b, L, dtype=torch.bool, device=DEV)
        t["reset"][:, 0] = True
        t["reset"][1, 400] = True
        clean = {k: None if v is None else v.clone() for k, v in t.items()}
        t["init_state"][0], t["init_state"][1] = nan, inf
        for k in ("x", "r", "i"):
            t[k][0, 300:] = nan
        t["x"][1, 250:400] = inf
        d2 = dout.clone()
        d2[0, 300:], d2[2] = nan, inf
        want, wf = ssd.ssd_glr_fwd(**clean)
        out = torch.zeros_like(want)
        _, fin = ssd.ssd_glr_fwd(**t, out=out)
        assert torch.equal(out[0, :300], want[0, :300]) and torch.equal(out[1, :250], want[1, :250])
        assert torch.equal(out[1, 400:], want[1, 400:]) and torch.equal(fin[:2], wf[:2])
        assert torch.equal(fin[2], t["init_state"][2]) and bool((out[0, 300:] == 0).all())
        gw = ssd.ssd_glr_bwd(**clean, dout=dout, dfinal_state=dfin)
        g = ssd.ssd_glr_bwd(**t, dout=d2, dfinal_state=dfin)
        for k in ("dx", "dr", "di"):
            assert torch.equal(g[k][0], gw[k][0]) and torch.equal(g[k][2], gw[k][2]), k
            assert torch.equal(g[k][1, 401:], gw[k][1, 401:]) and bool((g[k][0, 300:] == 0).all()), k
        assert bool((g["dinit"][:2] == 0).all()) and torch.equal(g["dinit"][2], dfin[2])


@pytest.mark.parametrize("dtype", [F32, BF], ids=["f32", "bf16"])
@pytest.mark.parametrize("b,D", [(1, 1), (3, 40), (5, 130), (300, 64), (2, 4100)])
def test_step(b, D, dtype):
    t, _, _ = make(b, 1, D, dtype, seed=b + D, layout="offset" if D == 130 else "fused", reset=0.3)
    h = host(t)
    f = glr_ref.forward(**h)
    state = t["init_state"].clone()
    args = [t["x"][:, 0], t["r"][:, 0], t["i"][:, 0], t["A"], t["r_bias"], t["i_bias"]]
    new = torch.full_like(state, float("nan"))
    out = ssd.ssd_glr_step(state, *args, reset=t["reset"][:, 0].contiguous(), new_state=new)
    assert torch.equal(state, t["init_state"])
    check("out", out, f["h"][:, 0], f["eh"][:, 0])
    check("state", new, f["fin"], f["efin"])
    out2 = ssd.ssd_glr_step(state, *args, reset=t["reset"][:, 0].contiguous())
    assert torch.equal(state, new) and torch.equal(out2, out)


def test_step_by_step_follows_the_scan():
    b, L, D = 3, 40, 200
    t, _, _ = make(b, L, D, BF, seed=8, reset=0.1)
    f = glr_ref.forward(**host(t))
    _, fin = ssd.ssd_glr_fwd(**t)
    st = t["init_state"].clone()
    for k in range(L):
        out = ssd.ssd_glr_step(st, t["x"][:, k], t["r"][:, k], t["i"][:, k], t["A"], t["r_bias"], t["i_bias"],
                               reset=t["reset"][:, k].contiguous())
        check("out %d" % k, out, f["h"][:, k], f["eh"][:, k])
    check("state", st, f["fin"], f["efin"])
    check("final", fin, f["fin"], f["efin"])


def test_a_sequence_in_two_calls_in_place():
    # the final state written over the initial one, with and without resets
    b, L, D, cut = 2, 1500, 72, 900
    for reset in (0.0, 0.003):
        t, _, _ = make(b, L, D, BF, seed=9, reset=reset)
        f = glr_ref.forward(**host(t))
        st = t["init_state"].clone()
        outs = []
        for lo, hi in ((0, cut), (cut, L)):
            part = {k: (v[:, lo:hi].contiguous() if k in ("x", "r", "i", "reset") and v is not None else v) for k, v in t.items()}
            part["init_state"] = st
            o, fin = ssd.ssd_glr_fwd(**part, final_state=st)
            assert fin is st
            outs.append(o)
        check("out", torch.cat(outs, 1), f["h"], f["eh"])
        check("state", st, f["fin"], f["efin"])


def test_repeats_are_bitwise_equal_and_ignore_the_workspace():
    b, L, D = 2, 4000, 192
    t, dout, dfin = make(b, L, D, BF, seed=10, reset=0.001)
    lib = ssd.lib()
    first = None
    for fill in (0, 255, 0x7F):
        ws = torch.full((ssd.ssd_glr_workspace(b, L, D, True),), fill, dtype=torch.uint8, device=DEV)
        out, fin, states = torch.empty_like(t["x"]), torch.empty(b, D, device=DEV), ssd.ssd_glr_states(t["x"])
        keep, d = ssd._descs(t["x"], t["r"], t["i"], t["A"], t["r_bias"], t["i_bias"], t["reset"], None,
                             t["init_state"], out, fin, states)
        assert lib.ssd_glr_fwd(*d, ws.data_ptr(), ws.numel(), torch.cuda.current_stream().cuda_stream) == 0
        g = ssd.ssd_glr_bwd(**t, dout=dout, dfinal_state=dfin, states=states)
        g2 = ssd.ssd_glr_bwd(**t, dout=dout, dfinal_state=dfin)
        got = [out, fin, states] + [g[k] for k in sorted(g)]
        for k in g:
            assert torch.equal(g[k], g2[k]), k
        if first is None:
            first = got
        for p, q in zip(got, first):
            assert torch.equal(p, q)


def test_gradients_against_differences():
    # <gradients, direction> of the kernel against the reference forward's
    # central difference along the direction
    b, L, D = 2, 333, 20
    t, dout, dfin = make(b, L, D, F32, seed=11, reset=0.01, lengths=[333, 200], amin=0.05)
    g = ssd.ssd_glr_bwd(**t, dout=dout, dfinal_state=dfin)
    h = host(t)
    rng = np.random.default_rng(12)
    do, df = dout.cpu().double().numpy(), dfin.cpu().double().numpy()

    def obj(a):
        f = glr_ref.forward(**a)
        return float((f["h"] * do).sum() + (f["fin"] * df).sum())

    for key, name in (("x", "dx"), ("r", "dr"), ("i", "di"), ("A", "dA"), ("rb", "dr_bias"), ("ib", "di_bias"), ("init", "dinit")):
        v = rng.standard_normal(h[key].shape) * (0.1 * np.abs(h[key]) if key == "A" else 1.0)
        eps = 1e-5
        d = (obj({**h, key: h[key] + eps * v}) - obj({**h, key: h[key] - eps * v})) / (2 * eps)
        p = g[name].cpu().double().numpy() * v
        # the difference's own error is of order eps^2; fp32 gradients carry a
        # few hundred U of each term (the bounds of the element-wise test)
        assert abs(p.sum() - d) <= 1e-4 * np.abs(p).sum() + 1e-6, (name, p.sum(), d)


def test_graph_replays_and_streams():
    b, L, D = 2, 1100, 128
    t, dout, dfin = make(b, L, D, BF, seed=13, reset=0.002)
    want, wf = ssd.ssd_glr_fwd(**t)
    wg = ssd.ssd_glr_bwd(**t, dout=dout, dfinal_state=dfin)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        ssd.ssd_glr_fwd(**t)
        ssd.ssd_glr_bwd(**t, dout=dout, dfinal_state=dfin)
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        states = ssd.ssd_glr_states(t["x"])
        out, fin = ssd.ssd_glr_fwd(**t, states=states)
        g = ssd.ssd_glr_bwd(**t, dout=dout, dfinal_state=dfin, states=states)
    for k in range(4):
        say("replay", k)
        for v in (out, fin, *g.values()):
            v.fill_(float("nan"))
        graph.replay()
        e, ef = ssd.ssd_glr_fwd(**t)  # eager work between the replays
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.equal(fin, wf) and torch.equal(e, want) and torch.equal(ef, wf)
        for n in wg:
            assert torch.equal(g[n], wg[n]), n
    # two streams at once, one of them given by its handle
    s2 = torch.cuda.Stream()
    s2.wait_stream(torch.cuda.current_stream())
    res = []
    for k in range(6):
        with torch.cuda.stream(s):
            res.append(ssd.ssd_glr_fwd(**t))
        res.append(ssd.ssd_glr_fwd(**t, stream=s2.cuda_stream))
    torch.cuda.synchronize()
    for o, f in res:
        assert torch.equal(o, want) and torch.equal(f, wf)


def test_the_default_stream_by_handle_and_two_host_threads():
    import threading
    b, L, D = 2, 600, 128
    t, dout, dfin = make(b, L, D, BF, seed=16, reset=0.002)
    want, wf = ssd.ssd_glr_fwd(**t)
    wg = ssd.ssd_glr_bwd(**t, dout=dout, dfinal_state=dfin)
    torch.cuda.synchronize()
    with torch.cuda.stream(torch.cuda.Stream()):
        out, fin = ssd.ssd_glr_fwd(**t, stream=torch.cuda.default_stream().cuda_stream)
    torch.cuda.synchronize()
    assert torch.equal(out, want) and torch.equal(fin, wf)
    bad = []

    def work():
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                for _ in range(20):
                    o, f = ssd.ssd_glr_fwd(**t)
                    g = ssd.ssd_glr_bwd(**t, dout=dout, dfinal_state=dfin)
                torch.cuda.current_stream().synchronize()
                if not (torch.equal(o, want) and torch.equal(f, wf) and all(torch.equal(g[k], wg[k]) for k in wg)):
                    bad.append("differs")
                torch.cuda.current_stream().synchronize()
        except Exception as e:  # reported below
            bad.append(repr(e))

    th = [threading.Thread(target=work) for _ in range(3)]
    for x in th:
        x.start()
    for x in th:
        x.join()
    assert not bad, bad


def test_far_offsets():
    # a batch stride beyond 2^31 elements, reached through views
    b, L, D = 2, 300, 64
    big = torch.empty((1 << 31) + (1 << 16), dtype=BF, device=DEV)
    x = big.as_strided((b, L, D), (1 << 31, D, 1))
    t, _, _ = make(b, L, D, BF, seed=14)
    x.copy_(t["x"])
    want, wf = ssd.ssd_glr_fwd(**t)
    t["x"] = x
    out, fin = ssd.ssd_glr_fwd(**t)
    assert torch.equal(out, want) and torch.equal(fin, wf)


def test_many_rows_and_a_wide_row():
    for b, L, D in ((70000, 1, 8), (1, 3, 70000)):
        t, _, _ = make(b, L, D, F32, seed=15)
        f = glr_ref.forward(**host(t))
        out, fin = ssd.ssd_glr_fwd(**t)
        check("out", out, f["h"], f["eh"])
        check("final", fin, f["fin"], f["efin"])


def test_a_very_long_row():
    # constant gates and input: h_t = g (1 - a^t) / (1 - a), g the input's share;
    # 8192 chunks forward, 16384 back, inputs of stride 0 along the row
    L, D = 1 << 20, 64
    one = torch.ones(1, 1, D, device=DEV)
    A = -torch.linspace(1e-4, 0.4, D, device=DEV)
    x, z = one.expand(1, L, D), torch.zeros(1, 1, D, device=DEV).expand(1, L, D)
    states = ssd.ssd_glr_states(x)
    out, fin = ssd.ssd_glr_fwd(x, z, z, A, states=states)
    a = np.exp(A.cpu().double().numpy() * 0.5)
    g = np.sqrt(-np.expm1(A.cpu().double().numpy())) * 0.5
    # The decay is off by ea U (2 + 8 |log a| and 8 for the roundings of a
    # step) and the input's share by 40 U; to first order in them h moves by
    # (ea |h| / (1 - a) + 40 |h|) U, as a sum of what every token adds
    for t in (1, 100, 128, 129, 4096, 500000, L):
        want = g * -np.expm1(t * np.log(a)) / (1 - a)
        tol = ((10 + 8 * np.abs(np.log(a))) / (1 - a) + 40) * glr_ref.U * want
        got = out[0, t - 1].cpu().double().numpy()
        assert np.all(np.abs(got - want) <= tol), (t, np.max(np.abs(got - want) / tol))
    # the final state goes by the chunks' maps, the last output by the tokens:
    # the same bound for either
    assert np.all(np.abs(fin[0].cpu().double().numpy() - want) <= tol)
    # backward with dout = 1: c_0 = sum over t >= 1 of a^t
    d = ssd.ssd_glr_bwd(x, z, z, A, dout=x, states=states)
    want = a * -np.expm1(L * np.log(a)) / (1 - a)
    tol = ((10 + 8 * np.abs(np.log(a))) / (1 - a) + 40) * glr_ref.U * want
    assert np.all(np.abs(d["dinit"][0].cpu().double().numpy() - want) <= tol)


def test_optional_arguments_and_shared_inputs():
    b, L, D = 2, 200, 66
    t, dout, dfin = make(b, L, D, F32, seed=17)
    h = host(t)
    # no initial state, no gradient of the final one, no biases
    bare = dict(t, init_state=None, r_bias=None, i_bias=None)
    out, fin = ssd.ssd_glr_fwd(**bare, return_final_state=False)
    assert fin is None
    ref = dict(h, init=None, rb=None, ib=None)
    f = glr_ref.forward(**ref)
    check("out", out, f["h"], f["eh"])
    pre = dict(dx=torch.empty_like(out), dA=torch.empty(D, device=DEV))
    g = ssd.ssd_glr_bwd(**bare, dout=dout, want_bias=False, want_init=False, out=pre)
    assert g["dx"] is pre["dx"] and g["dA"] is pre["dA"] and g["dr_bias"] is None and g["dinit"] is None
    gr = glr_ref.backward(**ref, dout=dout.cpu().double().numpy())
    for k in ("dx", "dr", "di", "dA"):
        check(k, g[k], gr[k], gr["e" + k])
    # lengths outside [0, L] count as the nearer end; any nonzero byte is a reset
    ln = torch.tensor([-5, 10 ** 9], dtype=torch.int32, device=DEV)
    rs = torch.zeros(b, L, dtype=torch.uint8, device=DEV)
    rs[1, 37] = 255
    out = torch.zeros_like(t["x"])
    _, fin = ssd.ssd_glr_fwd(**dict(t, lengths=ln, reset=rs), out=out)
    f = glr_ref.forward(**dict(h, lengths=np.array([0, L]), reset=rs.cpu().numpy()))
    check("out", out, f["h"], f["eh"])
    check("final", fin, f["fin"], f["efin"])
    # one tensor for the input and both gates
    out, fin = ssd.ssd_glr_fwd(t["x"], t["x"], t["x"], t["A"])
    f = glr_ref.forward(h["x"], h["x"], h["x"], h["A"])
    check("out", out, f["h"], f["eh"])


@pytest.mark.parametrize("dtype", [F32, BF], ids=["f32", "bf16"])
@pytest.mark.parametrize("b,L,D,lengths", [(1, 1, 8, None), (2, 17, 40, [17, 4]), (3, 65, 72, [65, 63, 1]),
                                           (2, 301, 66, [299, 301])])
def test_tokens_that_do_not_exist_pass_the_state_on(b, L, D, lengths, dtype):
    # odd row ends with biases of infinity (gates always open or always shut),
    # for small and for large decays
    for amin, amax in ((0.001, 0.4), (0.6, 3.0)):
        t, dout, dfin = make(b, L, D, dtype, seed=18 + L, lengths=lengths, reset=0.01 if L > 100 else 0,
                             amin=amin, amax=amax)
        t["r_bias"][::3] = float("inf")
        t["i_bias"][1::4] = float("inf")
        h = host(t)
        out = torch.zeros(b, L, D, dtype=dtype, device=DEV)
        _, fin = ssd.ssd_glr_fwd(**t, out=out)
        f = glr_ref.forward(**h)
        check("out", out, f["h"], f["eh"])
        check("final", fin, f["fin"], f["efin"])
        g = ssd.ssd_glr_bwd(**t, dout=dout, dfinal_state=dfin)
        ref = glr_ref.backward(**h, dout=dout.float().cpu().double().numpy(), dfin=dfin.cpu().double().numpy())
        for k in ("dx", "dr", "di", "dA", "dr_bias", "di_bias", "dinit"):
            check(k, g[k], ref[k], ref["e" + k])
        # an r of -infinity or of the lowest value outweighs a bias of +infinity
        one = dict(t, lengths=torch.ones(b, dtype=torch.int32, device=DEV))
        one["r_bias"] = torch.full_like(t["r_bias"], float("inf"))
        for low in (float("-inf"), torch.finfo(dtype).min):
            one["r"] = torch.full_like(t["r"], low)
            _, fin = ssd.ssd_glr_fwd(**dict(one, reset=None))
            assert torch.equal(fin, t["init_state"])
            st = t["init_state"].clone()
            ssd.ssd_glr_step(st, t["x"][:, 0], one["r"][:, 0], t["i"][:, 0], t["A"], one["r_bias"])
            assert torch.equal(st, t["init_state"])
        # gates always shut: the state stays as it is
        t["r_bias"][:] = float("-inf")
        out = torch.zeros(b, L, D, dtype=dtype, device=DEV)
        _, fin = ssd.ssd_glr_fwd(**dict(t, reset=None), out=out)
        assert torch.equal(fin, t["init_state"])


@pytest.mark.parametrize("dtype", [F32, BF], ids=["f32", "bf16"])
def test_nan_inputs_show_in_their_gradients(dtype):
    # a NaN in one token of one channel: the reference's NaNs, no more and no
    # fewer, for each of the inputs and the output's gradient (finite otherwise)
    b, L, D = 2, 100, 16
    for where in ("x", "r", "i", "dout"):
        t, dout, dfin = make(b, L, D, dtype, seed=19, reset=0.02)
        (dout if where == "dout" else t[where])[1, 40, 3] = float("nan")
        g = ssd.ssd_glr_bwd(**t, dout=dout, dfinal_state=dfin)
        with np.errstate(invalid="ignore"):
            ref = glr_ref.backward(**host(t), dout=dout.float().cpu().double().numpy(), dfin=dfin.cpu().double().numpy())
        for k in ("dx", "dr", "di", "dA", "dr_bias", "di_bias", "dinit"):
            got = np.isnan(g[k].float().cpu().numpy())
            assert np.array_equal(got, np.isnan(ref[k])), (where, k, np.argwhere(got != np.isnan(ref[k]))[:4])


@pytest.mark.parametrize("case", SHAPES, ids=["b%d_L%d_D%d_%s" % c[:4] for c in SHAPES])
def test_gradients_from_fp32_output_gradients(case):
    # bf16 inputs and the fp32 gradient of a later fp32 stage, as a strided view
    # where the case has one
    b, L, D, layout, reset, lengths, init = case
    t, _, dfin = make(b, L, D, BF, seed=2 * L + D, layout=layout, reset=reset, lengths=lengths, init=init)
    g = torch.Generator().manual_seed(L)
    dout = torch.randn(b, L, D + (3 if layout == "offset" else 0), generator=g).to(DEV)[..., :D]
    if layout == "time_major":
        dout = dout.transpose(0, 1).contiguous().transpose(0, 1)
    if layout == "broadcast":
        dout = dout[:, :1].expand(b, L, D)
    states = ssd.ssd_glr_states(t["x"])
    ssd.ssd_glr_fwd(**t, states=states)
    ref = glr_ref.backward(**host(t), dout=dout.cpu().double().numpy(), dfin=dfin.cpu().double().numpy())
    for saved in (states, None):
        got = ssd.ssd_glr_bwd(**t, dout=dout, dfinal_state=dfin, states=saved)
        assert got["dx"].dtype == BF and got["dA"].dtype == F32
        for k in ("dx", "dr", "di", "dA", "dr_bias", "di_bias", "dinit"):
            check(k, got[k], ref[k], ref["e" + k])


@pytest.mark.parametrize("dtype,ddtype", [(F32, F32), (BF, BF), (BF, F32)], ids=["f32", "bf16", "bf16_f32"])
def test_inputs_that_pass_the_caches_by(dtype, ddtype):
    # 64 rows that are views of one: 128 MB and more, every row as the first
    b, L, D = 64, 512, 700
    t, dout, dfin = make(1, L, D, dtype, seed=20, reset=0.01, init=False)
    dout = dout.to(ddtype)
    w = {k: v.expand(b, *v.shape[1:]) if k in ("x", "r", "i") else v for k, v in t.items()}
    w["reset"] = t["reset"].expand(b, L).contiguous()
    out, fin = ssd.ssd_glr_fwd(**w)
    g = ssd.ssd_glr_bwd(**w, dout=dout.expand(b, L, D), dfinal_state=dfin.expand(b, D).contiguous())
    h = host(t)
    f = glr_ref.forward(**h)
    ref = glr_ref.backward(**h, dout=dout.float().cpu().double().numpy(), dfin=dfin.cpu().double().numpy())
    check("out", out[:1], f["h"], f["eh"])
    check("final", fin[:1], f["fin"], f["efin"])
    for v in (out, fin, *(g[k] for k in ("dx", "dr", "di", "dinit"))):
        assert bool((v == v[:1]).all())
    for k in ("dx", "dr", "di", "dinit"):
        check(k, g[k][:1], ref[k], ref["e" + k])
    for k in ("dA", "dr_bias", "di_bias"):
        check(k, g[k], b * ref[k], b * ref["e" + k])


def test_no_parameter_gradients():
    # none of them wanted: no partial sums are formed, the rest is the same
    b, L, D = 3, 300, 40
    t, dout, dfin = make(b, L, D, BF, seed=21, lengths=[300, 70, 0])
    states = ssd.ssd_glr_states(t["x"])
    ssd.ssd_glr_fwd(**t, states=states)
    want = ssd.ssd_glr_bwd(**t, dout=dout, dfinal_state=dfin, states=states)
    ws = torch.full((ssd.ssd_glr_workspace(b, L, D, True),), 0xA5, dtype=torch.uint8, device=DEV)
    # behind the chain words [b, segments, 128] of 8 bytes and 16 more
    chain = b * 5 * 128 * 8 + 16
    for st in (states, None):
        out = [torch.empty_like(t["x"]) for _ in range(3)] + [None] * 3 + [torch.empty(b, D, device=DEV)]
        keep, d = ssd._descs(t["x"], t["r"], t["i"], t["A"], t["r_bias"], t["i_bias"], None, t["lengths"], t["init_state"],
                             st, dout, dfin, *out)
        assert ssd.lib().ssd_glr_bwd(*d, ws.data_ptr(), ws.numel(), torch.cuda.current_stream().cuda_stream) == 0
        for k, v in zip(("dx", "dr", "di", None, None, None, "dinit"), out):
            assert v is None or torch.equal(v, want[k]), k
        part = -(-chain // 256) * 256
        assert bool((ws[part:part + b * 5 * 3 * D * 4] == 0xA5).all())


@pytest.mark.parametrize("largest", [-0.4, -3.0], ids=["small_decays", "any_decay"])
def test_gradients_where_the_factor_is_zero(largest):
    # A of 0 and above: the factor sqrt(1 - a^2) is 0 and so is the gradient
    # through it, the one through a h_{t-1} stays
    b, L, D = 2, 200, 10
    t, dout, dfin = make(b, L, D, F32, seed=22, lengths=[200, 131], reset=0.01)
    t["A"][:] = torch.tensor([0.0, -0.0, 1e-3, 0.1, 1e-30, -1e-30, -1e-7, -1e-3, -0.2, largest], device=DEV)
    g = ssd.ssd_glr_bwd(**t, dout=dout, dfinal_state=dfin)
    ref = glr_ref.backward(**host(t), dout=dout.cpu().double().numpy(), dfin=dfin.cpu().double().numpy())
    assert np.all(ref["dx"][..., :5][~(host(t)["reset"] != 0)] == 0) and np.all(ref["dA"][:4] != 0)
    for k in ("dx", "dr", "di", "dA", "dr_bias", "di_bias", "dinit"):
        check(k, g[k], ref[k], ref["e" + k])
