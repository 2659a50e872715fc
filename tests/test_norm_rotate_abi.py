"""Norm and rotation on the host: the calls it refuses (before any launch) and
the 64-bit reference against autograd (CPU only)."""
import numpy as np
import pytest
import torch

import norm_rotate_ref as ref
from mamba_ssd_scan_05_amd import ssd

BF = torch.bfloat16


def args(b=2, L=5, Hq=4, Hk=2, N=32, dtype=BF):
    z = torch.zeros
    return dict(q=z(b, L, Hq, N, dtype=dtype), k=z(b, L, Hk, N, dtype=dtype), qw=z(N), kw=z(N), freqs=z(N // 2),
                pos=z(b, L, dtype=torch.int32), q_out=z(b, L, Hq, N, dtype=dtype), k_out=z(b, L, Hk, N, dtype=dtype))


def call(a, eps=1e-6, interleaved=0):
    keep, d = ssd._descs(*a.values())
    return ssd.lib().ssd_norm_rotate_fwd(*d, eps, interleaved, None), ssd.ssd_last_error()


FWD = [
    ("q_none", dict(q=None), 1), ("k_none", dict(k=None), 1), ("q_out_none", dict(q_out=None), 1),
    ("q_rank3", dict(q=torch.zeros(2, 5, 32, dtype=BF)), 2), ("k_batch", dict(k=torch.zeros(1, 5, 2, 32, dtype=BF)), 2),
    ("k_width", dict(k=torch.zeros(2, 5, 2, 16, dtype=BF)), 2), ("L_zero", dict(q=torch.zeros(2, 0, 4, 32, dtype=BF)), 2),
    ("weight_per_head", dict(qw=torch.zeros(4, 32)), 2), ("weight_short", dict(kw=torch.zeros(31)), 2),
    ("freqs_long", dict(freqs=torch.zeros(20)), 2), ("freqs_table", dict(freqs=torch.zeros(5, 16)), 2),
    ("freqs_empty", dict(freqs=torch.zeros(0)), 2),
    ("positions_shape", dict(pos=torch.zeros(5, dtype=torch.int32)), 2), ("out_heads", dict(k_out=torch.zeros(2, 5, 4, 32, dtype=BF)), 2),
    ("q_f16", dict(q=torch.zeros(2, 5, 4, 32, dtype=torch.float16)), 3), ("k_f32", dict(k=torch.zeros(2, 5, 2, 32)), 3),
    ("weight_bf16", dict(qw=torch.zeros(32, dtype=BF)), 3), ("freqs_f64", dict(freqs=torch.zeros(16, dtype=torch.float64)), 3),
    ("positions_f32", dict(pos=torch.zeros(2, 5)), 3), ("out_f32", dict(q_out=torch.zeros(2, 5, 4, 32)), 3),
    ("q_columns", dict(q=torch.zeros(2, 5, 32, 4, dtype=BF).transpose(2, 3)), 4),
    ("out_view", dict(q_out=torch.zeros(2, 5, 8, 32, dtype=BF)[:, :, ::2]), 4),
    ("positions_view", dict(pos=torch.zeros(2, 10, dtype=torch.int32)[:, ::2]), 4),
    ("npair_odd", dict(freqs=torch.zeros(6)), 5),
    ("N_12", dict(q=torch.zeros(2, 5, 4, 12, dtype=BF), k=torch.zeros(2, 5, 2, 12, dtype=BF)), 5),
    ("N_264", dict(q=torch.zeros(2, 5, 4, 264, dtype=BF), k=torch.zeros(2, 5, 2, 264, dtype=BF)), 5),
]


@pytest.mark.parametrize("change,want", [(c, w) for _, c, w in FWD], ids=[n for n, _, _ in FWD])
def test_forward_refuses(change, want):
    a = args()
    a.update(change)
    st, msg = call(a)
    assert st == want and msg, (st, msg)


def test_options_overlaps_and_sizes_refused():
    for kw in (dict(eps=-1.0), dict(eps=float("nan")), dict(eps=float("inf")), dict(interleaved=2)):
        assert call(args(), **kw)[0] == 5, kw
    a = args()
    a["q_out"] = a["q"]
    assert call(a)[0] == 6
    a = args(Hq=2)
    a["k_out"] = a["q_out"]
    assert call(a)[0] == 6
    a = args()
    proj = torch.zeros(2, 5, 8, 32, dtype=BF)
    a.update(q=proj[:, :, :4], k=proj[:, :, 4:6])
    st, msg = call(a)
    assert st == 4 and "device" in msg or "address" in msg, (st, msg)  # the views pass; CPU memory does not
    row = torch.zeros(1, 1, 1, 32, dtype=BF)
    a = args(1, 1, 1, 1)
    a.update(q=row.expand(1, (1 << 25) + 1, 7, 32), k=row.expand(1, (1 << 25) + 1, 2, 32))
    assert call(a)[0] == 5
    # heads-first caches: a head stride of 2^23 elements passes the checks
    far = torch.empty(1 << 24, dtype=BF).as_strided((2, 5, 2, 32), (160, 32, 1 << 23, 1))
    a = args(Hq=2)
    a.update(q=far)
    st, msg = call(a)
    assert st == 4 and ("device" in msg or "address" in msg), (st, msg)
    assert ssd.lib().ssd_norm_rotate_workspace(12) == -1 and ssd.lib().ssd_norm_rotate_workspace(128) == 1024 * 2 * 128 * 4


def bwd_args():
    a = args()
    a["dq_out"], a["dk_out"] = a.pop("q_out"), a.pop("k_out")
    a.update(dq=torch.zeros_like(a["q"]), dk=torch.zeros_like(a["k"]), dqw=torch.zeros(32), dkw=torch.zeros(32))
    return a


def call_bwd(a, ws=None):
    ws = torch.zeros(ssd.lib().ssd_norm_rotate_workspace(32), dtype=torch.uint8) if ws is None else ws
    keep, d = ssd._descs(*a.values())
    return ssd.lib().ssd_norm_rotate_bwd(*d, 1e-6, 0, ws.data_ptr(), ws.numel(), None), ssd.ssd_last_error()


BWD = [("dq_out_none", dict(dq_out=None), 1), ("dk_none", dict(dk=None), 1), ("dk_out_shape", dict(dk_out=torch.zeros(2, 5, 1, 32, dtype=BF)), 2),
       ("dqw_shape", dict(dqw=torch.zeros(16)), 2), ("dq_f32", dict(dq=torch.zeros(2, 5, 4, 32)), 3),
       ("dk_view", dict(dk=torch.zeros(2, 5, 4, 32, dtype=BF)[:, :, :2]), 4)]


@pytest.mark.parametrize("change,want", [(c, w) for _, c, w in BWD], ids=[n for n, _, _ in BWD])
def test_backward_refuses(change, want):
    a = bwd_args()
    a.update(change)
    st, msg = call_bwd(a)
    assert st == want and msg, (st, msg)


def test_backward_refuses_overlaps_and_small_workspaces():
    a = bwd_args()
    a["dq"] = a["dq_out"]
    assert call_bwd(a)[0] == 6
    a = bwd_args()
    a["dqw"] = a["dkw"]
    assert call_bwd(a)[0] == 6
    assert call_bwd(bwd_args(), torch.zeros(64, dtype=torch.uint8))[0] == 7


@pytest.mark.parametrize("interleaved", [0, 1])
@pytest.mark.parametrize("npair", [0, 4, 12])
def test_reference_against_autograd(interleaved, npair):
    g = np.random.default_rng(5 + npair)
    b, L, H, N = 2, 3, 2, 24
    x, w, dy = g.standard_normal((b, L, H, N)), g.standard_normal(N), g.standard_normal((b, L, H, N))
    pos, freqs = g.integers(-9, 100, (b, L)), g.random(npair) if npair else None
    tx, tw = torch.tensor(x, requires_grad=True), torch.tensor(w, requires_grad=True)
    y = tx * torch.rsqrt((tx * tx).mean(-1, keepdim=True) + 1e-3) * tw
    if npair:
        ang = torch.tensor(pos)[..., None, None] * torch.tensor(freqs)
        z = y[..., :2 * npair]
        p, q = (z[..., ::2], z[..., 1::2]) if interleaved else (z[..., :npair], z[..., npair:])
        p, q = p * ang.cos() - q * ang.sin(), p * ang.sin() + q * ang.cos()
        z = torch.stack([p, q], -1).flatten(-2) if interleaved else torch.cat([p, q], -1)
        y = torch.cat([z, y[..., 2 * npair:]], -1)
    (y * torch.tensor(dy)).sum().backward()
    got, _ = ref.forward(x, w, pos, freqs, 1e-3, interleaved)
    assert np.allclose(got, y.detach().numpy(), rtol=1e-12, atol=1e-13)
    d = ref.backward(x, w, pos, freqs, 1e-3, interleaved, dy, 0)
    assert np.allclose(d["dx"], tx.grad.numpy(), rtol=1e-10, atol=1e-12)
    assert np.allclose(d["dw"], tw.grad.numpy(), rtol=1e-10, atol=1e-12)


def test_backward_takes_fp32_output_gradients():
    # both f32 with bf16 q and k: only the CPU memory is refused
    f32 = lambda a, k: torch.zeros_like(a[k], dtype=torch.float32)  # noqa: E731
    a = bwd_args()
    a.update(dq_out=f32(a, "dq_out"), dk_out=f32(a, "dk_out"))
    st, msg = call_bwd(a)
    assert st == 4 and ("device" in msg or "address" in msg), (st, msg)
    for k in ("dq_out", "dk_out"):  # one of each
        a = bwd_args()
        a[k] = f32(a, k)
        st, msg = call_bwd(a)
        assert st == 3 and "dk_out" in msg, (k, st, msg)
    a = bwd_args()
    a.update({k: f32(a, k) for k in ("q", "k", "dq", "dk")})  # f32 q and bf16 gradients
    assert call_bwd(a)[0] == 3


def test_no_workspace_without_weight_gradients():
    a = bwd_args()
    a.update(dqw=None, dkw=None)
    keep, d = ssd._descs(*a.values())
    st = ssd.lib().ssd_norm_rotate_bwd(*d, 1e-6, 0, None, 0, None)
    assert st == 4 and ("device" in ssd.ssd_last_error() or "address" in ssd.ssd_last_error()), ssd.ssd_last_error()
    for k in ("dqw", "dkw"):  # one of them is wanted
        a = bwd_args()
        a[k] = None
        keep, d = ssd._descs(*a.values())
        assert ssd.lib().ssd_norm_rotate_bwd(*d, 1e-6, 0, None, 0, None) == 1
