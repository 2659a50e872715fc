"""Gated linear recurrence on the host: the calls it refuses (before any
launch, so CPU tensors do), its workspace sizes, and the 64-bit reference
against autograd and against differences (CPU only)."""
import numpy as np
import pytest
import torch

import glr_ref
from mamba_ssd_scan_05_amd import ssd

BF, F32 = torch.bfloat16, torch.float32


def fwd_args(b=2, L=300, D=24, dtype=BF):
    ns = -(-L // ssd.SSD_GLR_SEGMENT)
    return dict(x=torch.zeros(b, L, D, dtype=dtype), r=torch.zeros(b, L, D, dtype=dtype),
                i=torch.zeros(b, L, D, dtype=dtype), A=-torch.ones(D), r_bias=torch.zeros(D), i_bias=torch.zeros(D),
                reset=torch.zeros(b, L, dtype=torch.uint8), lengths=torch.zeros(b, dtype=torch.int32),
                init_state=torch.zeros(b, D), out=torch.zeros(b, L, D, dtype=dtype), final_state=torch.zeros(b, D),
                states=torch.zeros(b, ns, D))


def call_fwd(a, ws="auto"):
    x = a["x"]
    if isinstance(ws, str):
        ws = torch.zeros(max(16, ssd.ssd_glr_workspace(2, 300, 24)), dtype=torch.uint8)
    keep, d = ssd._descs(*(a[k] for k in ("x", "r", "i", "A", "r_bias", "i_bias", "reset", "lengths", "init_state",
                                          "out", "final_state", "states")))
    del x
    return ssd.lib().ssd_glr_fwd(*d, ws.data_ptr() if ws is not None else None,
                                 ws.numel() if ws is not None else 0, None), ssd.ssd_last_error()


FWD = [
    ("x_none", dict(x=None), 1), ("r_none", dict(r=None), 1), ("A_none", dict(A=None), 1), ("out_none", dict(out=None), 1),
    ("x_rank", dict(x=torch.zeros(2, 300, 2, 12, dtype=BF)), 2),
    ("L_zero", dict(x=torch.zeros(2, 0, 24, dtype=BF)), 2),
    ("D_zero", dict(x=torch.zeros(2, 300, 0, dtype=BF)), 2),
    ("r_short", dict(r=torch.zeros(2, 299, 24, dtype=BF)), 2),
    ("i_broadcast_width", dict(i=torch.zeros(2, 300, 1, dtype=BF)), 2),
    ("A_per_state", dict(A=torch.zeros(24, 16)), 2), ("bias_shape", dict(r_bias=torch.zeros(23)), 2),
    ("reset_shape", dict(reset=torch.zeros(2, 299, dtype=torch.uint8)), 2),
    ("lengths_shape", dict(lengths=torch.zeros(3, dtype=torch.int32)), 2),
    ("states_shape", dict(states=torch.zeros(2, 2, 24)), 2), ("init_shape", dict(init_state=torch.zeros(2, 25)), 2),
    ("x_f16", dict(x=torch.zeros(2, 300, 24, dtype=torch.float16)), 3),
    ("x_int", dict(x=torch.zeros(2, 300, 24, dtype=torch.int32)), 3),
    ("r_f32", dict(r=torch.zeros(2, 300, 24)), 3), ("A_bf16", dict(A=torch.zeros(24, dtype=BF)), 3),
    ("reset_i32", dict(reset=torch.zeros(2, 300, dtype=torch.int32)), 3),
    ("lengths_i64", dict(lengths=torch.zeros(2, dtype=torch.int64)), 3),
    ("out_f32", dict(out=torch.zeros(2, 300, 24)), 3),
    ("x_transposed", dict(x=torch.zeros(2, 24, 300, dtype=BF).transpose(1, 2)), 4),
    ("out_view", dict(out=torch.zeros(2, 300, 48, dtype=BF)[..., :24]), 4),
    ("reset_view", dict(reset=torch.zeros(2, 600, dtype=torch.uint8)[:, ::2]), 4),
    ("x_wide_stride", dict(x=lambda: torch.empty(300 * ((1 << 22) + 8), dtype=BF).as_strided((1, 300, 24), (0, (1 << 22) + 8, 1)).expand(2, 300, 24)), 5),
]


@pytest.mark.parametrize("change,want", [(c, w) for _, c, w in FWD], ids=[n for n, _, _ in FWD])
def test_forward_refuses(change, want):
    a = fwd_args()
    a.update({k: v() if callable(v) else v for k, v in change.items()})
    st, msg = call_fwd(a)
    assert st == want and msg, (st, msg)


def test_forward_refuses_overlaps():
    for out, other in (("out", "x"), ("final_state", "states"), ("states", "init_state"), ("out", "i")):
        a = fwd_args(dtype=F32)
        n = max(a[out].numel(), a[other].numel())
        buf = torch.zeros(n + 4)
        a[out] = buf[:a[out].numel()].view(a[out].shape)
        a[other] = buf[4:4 + a[other].numel()].view(a[other].shape)
        st, msg = call_fwd(a)
        assert st == 6 and "overlaps" in msg, (out, other, st, msg)
    a = fwd_args()
    a["final_state"] = a["init_state"]  # exactly the initial state is fine; CPU memory is then refused
    st, msg = call_fwd(a)
    assert st == 4 and "address" in msg or "device" in msg, (st, msg)
    a = fwd_args()
    proj = torch.zeros(2, 300, 96, dtype=BF)
    a.update(x=proj[..., :24], r=proj[..., 24:48], i=proj[..., 48:72])
    a["final_state"] = proj.view(torch.float32)[0, :2, :24].contiguous()
    st, msg = call_fwd(a)
    assert st == 4, (st, msg)  # views are taken; only the CPU memory is refused


def test_workspace_checks():
    need = ssd.ssd_glr_workspace(2, 300, 24)
    assert need >= 2 * 2 * 64 * 8
    assert ssd.ssd_glr_workspace(2, 64, 24) == 0
    assert ssd.ssd_glr_workspace(2, 64, 24, backward=True) > 0
    assert ssd.ssd_glr_workspace(0, 256, 24) == -1 and ssd.ssd_glr_workspace(1, (1 << 24) + 1, 24) == -1
    assert ssd.ssd_glr_workspace(1 << 22, 1, 65) == -1
    st, msg = call_fwd(fwd_args(), ws=None)
    assert st == 1 and "workspace" in msg
    st, msg = call_fwd(fwd_args(), ws=torch.zeros(need - 1, dtype=torch.uint8))
    assert st == 7 and "workspace" in msg
    st, msg = call_fwd(fwd_args(), ws=torch.zeros(need + 16, dtype=torch.uint8)[1:])
    assert st == 4 and "workspace" in msg
    a = fwd_args()
    buf = torch.zeros(need + 8192, dtype=torch.uint8)
    a["final_state"] = buf[:2 * 24 * 4].view(torch.float32).view(2, 24)
    st, msg = call_fwd(a, ws=buf)
    assert st == 6 and "workspace overlaps final_state" in msg


def bwd_args(b=2, L=300, D=24, dtype=BF):
    a = fwd_args(b, L, D, dtype)
    del a["out"], a["final_state"]
    a.update(dout=torch.zeros(b, L, D, dtype=dtype), dfinal=torch.zeros(b, D),
             **{k: torch.zeros(b, L, D, dtype=dtype) for k in ("dx", "dr", "di")},
             **{k: torch.zeros(D) for k in ("dA", "drb", "dib")}, dinit=torch.zeros(b, D))
    return a


def call_bwd(a):
    ws = torch.zeros(ssd.ssd_glr_workspace(2, 300, 24, backward=True), dtype=torch.uint8)
    keep, d = ssd._descs(*(a[k] for k in ("x", "r", "i", "A", "r_bias", "i_bias", "reset", "lengths", "init_state",
                                          "states", "dout", "dfinal", "dx", "dr", "di", "dA", "drb", "dib", "dinit")))
    return ssd.lib().ssd_glr_bwd(*d, ws.data_ptr(), ws.numel(), None), ssd.ssd_last_error()


BWD = [
    ("dout_none", dict(dout=None), 1), ("dx_none", dict(dx=None), 1), ("di_none", dict(di=None), 1),
    ("dout_shape", dict(dout=torch.zeros(2, 300, 23, dtype=BF)), 2), ("states_shape", dict(states=torch.zeros(2, 1, 24)), 2),
    ("dA_shape", dict(dA=torch.zeros(1)), 2), ("dr_f32", dict(dr=torch.zeros(2, 300, 24)), 3),
    ("dinit_bf16", dict(dinit=torch.zeros(2, 24, dtype=BF)), 3),
    ("dx_view", dict(dx=torch.zeros(2, 300, 48, dtype=BF)[..., :24]), 4),
]


@pytest.mark.parametrize("change,want", [(c, w) for _, c, w in BWD], ids=[n for n, _, _ in BWD])
def test_backward_refuses(change, want):
    a = bwd_args()
    a.update(change)
    st, msg = call_bwd(a)
    assert st == want and msg, (st, msg)


def test_backward_refuses_overlaps():
    for p, q in (("dx", "dout"), ("dx", "dr"), ("dA", "drb"), ("dinit", "dfinal")):
        a = bwd_args()
        a[p] = a[q]
        st, msg = call_bwd(a)
        assert st == 6, (p, q, st, msg)


def step_args(b=3, D=24, dtype=BF):
    return dict(state=torch.zeros(b, D), x=torch.zeros(b, D, dtype=dtype), r=torch.zeros(b, D, dtype=dtype),
                i=torch.zeros(b, D, dtype=dtype), A=-torch.ones(D), r_bias=None, i_bias=None,
                reset=torch.zeros(b, dtype=torch.uint8), new_state=torch.zeros(b, D), out=torch.zeros(b, D, dtype=dtype))


STEP = [
    ("state_none", dict(state=None), 1), ("x_rank3", dict(x=torch.zeros(3, 1, 24, dtype=BF)), 2),
    ("b_zero", dict(x=torch.zeros(0, 24, dtype=BF)), 2), ("state_shape", dict(state=torch.zeros(3, 23)), 2),
    ("state_bf16", dict(state=torch.zeros(3, 24, dtype=BF)), 3), ("reset_shape", dict(reset=torch.zeros(4, dtype=torch.uint8)), 2),
    ("out_f32", dict(out=torch.zeros(3, 24)), 3), ("state_view", dict(state=torch.zeros(3, 48)[:, ::2]), 4),
]


@pytest.mark.parametrize("change,want", [(c, w) for _, c, w in STEP], ids=[n for n, _, _ in STEP])
def test_step_refuses(change, want):
    a = step_args()
    a.update(change)
    keep, d = ssd._descs(*a.values())
    st = ssd.lib().ssd_glr_step(*d, None)
    assert st == want and ssd.ssd_last_error(), (st, ssd.ssd_last_error())


def test_step_refuses_overlaps():
    a = step_args(dtype=F32)
    a["out"] = a["new_state"]
    keep, d = ssd._descs(*a.values())
    assert ssd.lib().ssd_glr_step(*d, None) == 6
    a = step_args(dtype=F32)
    a["new_state"] = a["x"]
    keep, d = ssd._descs(*a.values())
    assert ssd.lib().ssd_glr_step(*d, None) == 6


# --------------------------------------------------------------------------
# the reference itself
# --------------------------------------------------------------------------
def draw(b, L, D, seed, reset=True, lengths=True):
    g = np.random.default_rng(seed)
    n = lambda *s: g.standard_normal(s)  # noqa: E731
    return dict(x=n(b, L, D), r=n(b, L, D), i=n(b, L, D), A=-g.uniform(0.01, 2.0, D), rb=n(D), ib=n(D),
                reset=(g.random((b, L)) < 0.2).astype(np.uint8) if reset else None,
                lengths=g.integers(0, L + 1, b) if lengths else None, init=n(b, D)), n(b, L, D), n(b, D)


def test_reference_against_autograd():
    a, dout, dfin = draw(4, 13, 3, seed=1)
    ref = glr_ref.backward(**a, dout=dout, dfin=dfin)
    t = {k: torch.tensor(v) if k in ("reset", "lengths") else torch.tensor(v, requires_grad=True) for k, v in a.items()}
    h = t["init"]
    tot, hs = 0.0, []
    for k in range(13):
        s = torch.sigmoid(t["r"][:, k] + t["rb"])
        la = t["A"] * s
        keep = (t["reset"][:, k] == 0)[:, None]
        n = torch.where(keep, torch.exp(la) * h + torch.sqrt(-torch.expm1(2 * la)) * torch.sigmoid(t["i"][:, k] + t["ib"]) * t["x"][:, k],
                        torch.sigmoid(t["i"][:, k] + t["ib"]) * t["x"][:, k])
        ok = (k < t["lengths"])[:, None]
        h = torch.where(ok, n, h)
        hs.append(torch.where(ok, h, torch.zeros_like(h)))
        tot = tot + (torch.tensor(dout[:, k]) * hs[-1]).sum()
    tot = tot + (torch.tensor(dfin) * h).sum()
    tot.backward()
    f = glr_ref.forward(**a)
    assert np.allclose(f["h"], torch.stack(hs, 1).detach().numpy(), rtol=1e-12, atol=1e-13)
    assert np.allclose(f["fin"], h.detach().numpy(), rtol=1e-12, atol=1e-13)
    for name, key in (("dx", "x"), ("dr", "r"), ("di", "i"), ("dA", "A"), ("dr_bias", "rb"), ("di_bias", "ib"), ("dinit", "init")):
        assert np.allclose(ref[name], t[key].grad.numpy(), rtol=1e-10, atol=1e-12), name


def test_reference_bound_holds_for_a_plain_fp32_evaluation():
    # an fp32 evaluation token by token stays inside the bound, and the bound
    # is no more than a few hundred times what is lost
    a, _, _ = draw(2, 200, 16, seed=2)
    f32 = {k: (v.astype(np.float32) if v is not None and v.dtype == np.float64 else v) for k, v in a.items()}
    f = glr_ref.forward(**{k: (v.astype(np.float64) if v is not None and v.dtype == np.float32 else v) for k, v in f32.items()})
    one = np.float32(1)
    h = f32["init"].copy()
    worst = 0.0
    for k in range(200):
        s = one / (one + np.exp(-(f32["r"][:, k] + f32["rb"])))
        la = f32["A"] * s
        u = f32["x"][:, k] / (one + np.exp(-(f32["i"][:, k] + f32["ib"])))
        n = np.where(f32["reset"][:, k, None] != 0, u, np.exp(la) * h + np.sqrt(-np.expm1(2 * la)) * u)
        ok = (k < f32["lengths"])[:, None]
        h = np.where(ok, n, h)
        err = np.where(ok, np.abs(h - f["h"][:, k]), 0)
        assert np.all(err <= f["eh"][:, k])
        worst = max(worst, float((err / np.maximum(f["eh"][:, k], 1e-30)).max()))
    assert 0.003 < worst <= 1.0, worst


def test_backward_takes_fp32_output_gradients():
    # f32 dout with bf16 inputs passes the checks (only the CPU memory is
    # refused); bf16 with f32 inputs does not, nor any other mixture
    a = bwd_args()
    a["dout"] = torch.zeros(2, 300, 24)
    st, msg = call_bwd(a)
    assert st == 4 and ("device" in msg or "address" in msg), (st, msg)
    a = bwd_args(dtype=F32)
    a["dout"] = torch.zeros(2, 300, 24, dtype=BF)
    st, msg = call_bwd(a)
    assert st == 3 and "dout" in msg, (st, msg)
    for k in ("r", "dx", "di"):
        a = bwd_args()
        a[k] = torch.zeros(2, 300, 24)
        assert call_bwd(a)[0] == 3, k
    a = bwd_args()
    a["dout"] = torch.zeros(2, 300, 24, dtype=torch.float16)
    assert call_bwd(a)[0] == 3


def test_the_initial_state_in_place_passes_the_overlap_check():
    a = fwd_args()
    a["final_state"] = a["init_state"]
    st, msg = call_fwd(a)
    assert st == 4 and ("address" in msg or "device" in msg), (st, msg)  # only the CPU memory is refused
