"""The paged cache and the attention over it on the host: the calls they refuse
(before any launch), and the 64-bit reference against autograd-free torch (CPU only)."""
import numpy as np
import pytest
import torch

import attn_ref as ref
from mamba_ssd_scan_05_amd import ssd

BF = torch.bfloat16
I32 = torch.int32


def z(*s, dtype=BF):
    return torch.zeros(s, dtype=dtype)


def append_args(b=2, L=3, Hq=4, Hk=2, N=32, pages=5, size=8, width=3):
    return dict(q=z(b, L, Hq, N), k=z(b, L, Hk, N), v=z(b, L, Hk, N), freqs=z(N // 2, dtype=torch.float32),
                page_table=z(b, width, dtype=I32), start=z(b, dtype=I32), tokens=z(b, dtype=I32), q_out=z(b, L, Hq, N),
                k_cache=z(pages, size, Hk, N), v_cache=z(pages, size, Hk, N))


def append(a, interleaved=0):
    keep, d = ssd._descs(*a.values())
    return ssd.lib().ssd_kv_append(*d, interleaved, None), ssd.ssd_last_error()


def passes(st, msg):
    """Every check but the last: CPU memory is no device memory."""
    return st == 4 and ("device" in msg or "address" in msg)


far = torch.empty(1 << 26, dtype=BF)  # never touched
APPEND = [
    ("k_none", dict(k=None), 1), ("v_none", dict(v=None), 1), ("table_none", dict(page_table=None), 1),
    ("start_none", dict(start=None), 1), ("k_cache_none", dict(k_cache=None), 1), ("v_cache_none", dict(v_cache=None), 1),
    ("q_without_q_out", dict(q_out=None), 1), ("q_out_without_q", dict(q=None), 1),
    ("k_rank", dict(k=z(2, 3, 64)), 2), ("q_rank", dict(q=z(2, 3, 128)), 2), ("v_heads", dict(v=z(2, 3, 1, 32)), 2),
    ("q_width", dict(q=z(2, 3, 4, 16)), 2), ("no_tokens", dict(k=z(2, 0, 2, 32)), 2), ("cache_rank", dict(k_cache=z(40, 2, 32)), 2),
    ("cache_heads", dict(k_cache=z(5, 8, 4, 32)), 2), ("caches_differ", dict(v_cache=z(6, 8, 2, 32)), 2),
    ("empty_cache", dict(k_cache=z(0, 8, 2, 32)), 2), ("table_rank", dict(page_table=z(6, dtype=I32)), 2),
    ("table_batch", dict(page_table=z(3, 3, dtype=I32)), 2), ("table_empty", dict(page_table=z(2, 0, dtype=I32)), 2),
    ("start_batch", dict(start=z(3, dtype=I32)), 2), ("tokens_per_token", dict(tokens=z(2, 3, dtype=I32)), 2),
    ("freqs_long", dict(freqs=z(20, dtype=torch.float32)), 2), ("q_out_heads", dict(q_out=z(2, 3, 2, 32)), 2),
    ("k_f16", dict(k=z(2, 3, 2, 32, dtype=torch.float16)), 3), ("v_f32", dict(v=z(2, 3, 2, 32, dtype=torch.float32)), 3),
    ("cache_f32", dict(k_cache=z(5, 8, 2, 32, dtype=torch.float32)), 3), ("table_i64", dict(page_table=z(2, 3, dtype=torch.int64)), 3),
    ("start_i64", dict(start=z(2, dtype=torch.int64)), 3), ("tokens_u8", dict(tokens=z(2, dtype=torch.uint8)), 3),
    ("freqs_bf16", dict(freqs=z(16)), 3), ("q_out_view", dict(q_out=z(2, 3, 8, 32)[:, :, ::2]), 4),
    ("cache_columns", dict(k_cache=z(5, 8, 32, 2).transpose(2, 3)), 4),
    ("cache_unaligned", dict(k_cache=z(5 * 8 * 2 * 32 + 8)[4:5 * 8 * 2 * 32 + 4].view(5, 8, 2, 32)), 4),
    ("cache_row_stride", dict(v_cache=z(5, 8, 2, 36)[..., :32]), 4), ("cache_one_page", dict(k_cache=z(1, 8, 2, 32).expand(5, 8, 2, 32)), 4),
    ("cache_rows_overlap", dict(k_cache=far.as_strided((5, 8, 2, 32), (512, 64, 16, 1))), 4),
    ("start_view", dict(start=z(4, dtype=I32)[::2]), 4), ("table_columns", dict(page_table=z(3, 2, dtype=I32).t()), 4),
    ("npair_odd", dict(freqs=z(6, dtype=torch.float32)), 5), ("cache_slot_stride", dict(k_cache=far.as_strided((2, 2, 2, 32), (1 << 25, (1 << 24) + 8, 32, 1)),
                                                                                        v_cache=z(2, 2, 2, 32)), 5),
]


@pytest.mark.parametrize("change,want", [(c, w) for _, c, w in APPEND], ids=[n for n, _, _ in APPEND])
def test_append_refuses(change, want):
    a = append_args()
    a.update(change)
    st, msg = append(a)
    assert st == want and msg and not passes(st, msg), (st, msg)


def test_append_sizes_and_options_refused():
    assert append(append_args(), 2)[0] == 5
    for N in (12, 264):
        assert append(append_args(N=N))[0] == 5
    a = append_args(b=1, L=1, pages=1, size=1 << 11, width=1 << 20)
    st, msg = append(a)
    assert st == 5 and "too many" in msg, (st, msg)
    row = torch.zeros(1, 1, 1, 8, dtype=BF)
    a = append_args(1, 1, 1, 1, 8)
    a.update(q=row.expand(1, (1 << 24) + 1, 1, 8), k=row.expand(1, (1 << 24) + 1, 1, 8))
    assert append(a)[0] == 5


def test_strides_of_pages():
    # a page stride just below 2^32 elements passes, one of 2^32 does not
    import ctypes
    for stride, ok in (((1 << 32) - 8, True), (1 << 32, False)):
        a = append_args()
        keep, d = ssd._descs(*a.values())
        d = list(d)
        for i in (8, 9):
            p = ssd.describe(a["k_cache" if i == 8 else "v_cache"])
            p.contents.data = (1 << 44) * (i - 6)  # far from each other, never touched
            p.contents.strides[0] = stride
            d[i] = ctypes.cast(p, ctypes.c_void_p)
        st = ssd.lib().ssd_kv_append(*d, 0, None)
        assert (st == 4 and passes(st, ssd.ssd_last_error())) if ok else st == 5, (st, ssd.ssd_last_error())


def test_append_takes_what_is_documented():
    assert passes(*append(append_args()))
    a = append_args()
    a.update(q=None, q_out=None, tokens=None, freqs=None)
    assert passes(*append(a))
    proj, wide = z(2, 3, 8, 32), z(2, 9, dtype=I32)
    both, inner = z(5, 2, 8, 2, 32), z(5, 8, 2, 2, 32)
    heads = z(5, 2, 8, 32)
    a = append_args()
    a.update(q=proj[:, :, :4], k=proj[:, :, 4:6], v=proj[:, :, 6:], page_table=wide[:, 2:5])
    assert passes(*append(a))
    for k, v in ((both[:, 0], both[:, 1]), (both[:, 1], both[:, 0]), (inner[:, :, 0], inner[:, :, 1]),
                 (heads.transpose(1, 2), z(5, 2, 8, 32).transpose(1, 2)),
                 (z(5, 8, 2, 64)[..., :32], z(5, 8, 2, 64)[..., 32:]), (z(10, 8, 2, 32)[:5], z(10, 8, 2, 32)[5:])):
        a.update(k_cache=k, v_cache=v)
        assert passes(*append(a)), (k.stride(), v.stride())
    t = z(5, 8, 2, 64)
    a.update(k_cache=t[..., :32], v_cache=t[..., 32:])
    assert passes(*append(a))


def test_append_overlaps_refused():
    a = append_args()
    a["v_cache"] = a["k_cache"]
    assert append(a)[0] == 6
    buf = z(11 * 8 * 2 * 32)
    a.update(k_cache=buf[:5 * 512].view(5, 8, 2, 32), v_cache=buf[4 * 512:9 * 512].view(5, 8, 2, 32))
    assert append(a)[0] == 6
    # in each other's gaps, but for a part: rows of 32 at a distance of 16
    t = z(5, 8, 2, 64)
    a.update(k_cache=t[..., :32], v_cache=t[..., 16:48])
    assert append(a)[0] == 6
    # the second's last page reaches into the first's next page
    both = z(6, 2, 8, 2, 32).view(-1)
    st = (1024, 64, 32, 1)
    a.update(k_cache=both.as_strided((5, 8, 2, 32), st), v_cache=both[768:].as_strided((5, 8, 2, 32), st))
    assert append(a)[0] == 6
    for name in ("q_out", "q", "k", "v"):
        a = append_args(Hq=2)
        if name == "q_out":
            a["q_out"] = a["q"]
        else:
            a[name] = a["k_cache"].view(-1)[:2 * 3 * 2 * 32].view(2, 3, 2, 32)
        assert append(a)[0] == 6, name


def attn_args(b=2, L=3, Hq=4, Hk=2, N=32, pages=5, size=8, width=3, step=False):
    q = (b, Hq, N) if step else (b, L, Hq, N)
    a = dict(q=z(*q), k_cache=z(pages, size, Hk, N), v_cache=z(pages, size, Hk, N), page_table=z(b, width, dtype=I32),
             start=z(b, dtype=I32), tokens=z(b, dtype=I32), out=z(*q), lse=z(*q[:-1], dtype=torch.float32))
    if step:
        del a["tokens"]
    return a


def attn(a, scale=0.5, window=0, ws=None, ws_bytes=None):
    step = "tokens" not in a
    if ws is None:
        ws = torch.zeros(1 << 23, dtype=torch.uint8)
    keep, d = ssd._descs(*a.values())
    f = ssd.lib().ssd_attn_step if step else ssd.lib().ssd_attn_fwd
    return f(*d, scale, window, ws.data_ptr(), ws.numel() if ws_bytes is None else ws_bytes, None), ssd.ssd_last_error()


ATTN = [
    ("q_none", dict(q=None), 1), ("k_cache_none", dict(k_cache=None), 1), ("v_cache_none", dict(v_cache=None), 1),
    ("table_none", dict(page_table=None), 1), ("start_none", dict(start=None), 1), ("out_none", dict(out=None), 1),
    ("q_rank", dict(q=z(6, 4, 32)), 2), ("cache_rank", dict(k_cache=z(5, 8, 64)), 2), ("cache_width", dict(k_cache=z(5, 8, 2, 64)), 2),
    ("heads_do_not_divide", dict(k_cache=z(5, 8, 3, 32), v_cache=z(5, 8, 3, 32)), 2), ("v_pages", dict(v_cache=z(4, 8, 2, 32)), 2),
    ("table_batch", dict(page_table=z(1, 3, dtype=I32)), 2), ("out_shape", dict(out=z(2, 3, 2, 32)), 2),
    ("lse_per_key_head", dict(lse=z(2, 3, 2, dtype=torch.float32)), 2), ("tokens_batch", dict(tokens=z(3, dtype=I32)), 2),
    ("q_f32", dict(q=z(2, 3, 4, 32, dtype=torch.float32)), 3), ("out_f32", dict(out=z(2, 3, 4, 32, dtype=torch.float32)), 3),
    ("lse_bf16", dict(lse=z(2, 3, 4)), 3), ("start_i64", dict(start=z(2, dtype=torch.int64)), 3),
    ("q_columns", dict(q=z(2, 3, 32, 4).transpose(2, 3)), 4), ("out_view", dict(out=z(2, 3, 8, 32)[:, :, ::2]), 4),
    ("out_unaligned", dict(out=z(2 * 3 * 4 * 32 + 8)[4:-4].view(2, 3, 4, 32)), 4),
    ("cache_unaligned", dict(v_cache=z(5 * 8 * 2 * 32 + 8)[4:-4].view(5, 8, 2, 32)), 4),
]


@pytest.mark.parametrize("change,want", [(c, w) for _, c, w in ATTN], ids=[n for n, _, _ in ATTN])
def test_attention_refuses(change, want):
    a = attn_args()
    a.update(change)
    st, msg = attn(a)
    assert st == want and msg and not passes(st, msg), (st, msg)


def test_attention_options_and_sizes_refused():
    for s in (0.0, float("nan"), float("inf"), 1e-39):
        assert attn(attn_args(), scale=s)[0] == 5, s
    assert attn(attn_args(), window=-1)[0] == 5
    assert attn(attn_args(N=12))[0] == 5 and attn(attn_args(N=264))[0] == 5
    assert ssd.ssd_attn_workspace(0, 1, 4, 2, 64) == -1 and ssd.ssd_attn_workspace(1, 1, 5, 2, 64) == -1
    assert ssd.ssd_attn_workspace(1, 1, 4, 2, 60) == -1 and ssd.ssd_attn_workspace(1 << 17, 1, 4, 2, 64) == -1
    assert ssd.ssd_attn_workspace(1, 1 << 24, 128, 1, 64) == -1 and ssd.ssd_attn_workspace(1, 1, 4, 2, 64) > 0
    # far more rows than the device holds at once need no workspace
    assert ssd.ssd_attn_workspace(1 << 16, 1, 8, 8, 64) == 0
    a = attn_args(b=1, L=1, pages=1, size=1 << 11, width=1 << 20)
    assert attn(a)[0] == 5


def test_attention_takes_what_is_documented():
    for s in (False, True):
        a = attn_args(step=s)
        assert passes(*attn(a, scale=-0.5, window=1 << 40))
        a["lse"] = None
        assert passes(*attn(a))
    a = attn_args()
    proj = z(2, 3, 8, 32)
    kv = z(5, 2, 8, 2, 32)
    a.update(tokens=None, q=proj[:, :, 1:5], k_cache=kv[:, 0], v_cache=kv[:, 1], page_table=z(2, 9, dtype=I32)[:, 1:4])
    assert passes(*attn(a))
    a.update(k_cache=kv[:, 0], v_cache=kv[:, 0])  # an input may be two of them
    assert passes(*attn(a))
    a.update(k_cache=z(1, 8, 2, 32).expand(5, 8, 2, 32))  # and be read at one place for all
    assert passes(*attn(a))


def test_attention_overlaps_and_workspaces_refused():
    for name in ("q", "k_cache"):
        a = attn_args()
        a["out"] = a[name].view(-1)[:2 * 3 * 4 * 32].view(2, 3, 4, 32)
        assert attn(a)[0] == 6, name
    a = attn_args()
    a["lse"] = a["out"].view(-1).view(torch.float32)[:24].view(2, 3, 4)
    assert attn(a)[0] == 6
    a = attn_args()
    need = ssd.ssd_attn_workspace(2, 3, 4, 2, 32)
    ws = torch.zeros(need + 16, dtype=torch.uint8)
    assert passes(*attn(a, ws=ws[:need]))
    assert attn(a, ws=ws, ws_bytes=need - 1)[0] == 7
    assert attn(a, ws=ws[8:])[0] == 4 and "aligned" in ssd.ssd_last_error()
    a["out"] = ws[:2 * 3 * 4 * 32 * 2].view(BF).view(2, 3, 4, 32)
    assert attn(a, ws=ws)[0] == 6
    a = attn_args()
    keep, d = ssd._descs(*a.values())
    assert ssd.lib().ssd_attn_fwd(*d, 0.5, 0, None, 0, None) == 1


@pytest.mark.parametrize("window", [0, 3])
def test_reference_against_a_softmax(window):
    g = np.random.default_rng(3)
    q, k, v = g.standard_normal((4, 8)), g.standard_normal((9, 8)), g.standard_normal((9, 8))
    k[2] = np.nan  # on no page
    pos = np.array([8, 5, 0, -1])
    out, lse, eo, el = ref.attend(q, k, v, pos, 0.7, window, 0.0)
    for i, p in enumerate(pos):
        j = [x for x in range(9) if x <= p and x != 2 and (not window or x > p - window)]
        if not j:
            assert (out[i] == 0).all() and lse[i] == -np.inf and (eo[i] == 0).all()
            continue
        s = torch.tensor(0.7 * k[j] @ q[i])
        assert np.allclose(out[i], torch.softmax(s, 0).numpy() @ v[j], rtol=1e-13, atol=1e-13)
        assert np.isclose(lse[i], torch.logsumexp(s, 0).item(), rtol=1e-13)
        # what a rounding to fp32 changes lies within the bound
        assert np.abs(out[i] - out[i].astype(np.float32)).max() < eo[i].min() < 1e-4 and el[i] < 1e-4


@pytest.mark.parametrize("interleaved", [False, True])
def test_reference_turn_against_complex_numbers(interleaved):
    g = np.random.default_rng(4)
    x, pos, f = g.standard_normal((3, 2, 12)), np.array([[0], [7], [1 << 20]]), g.random(4)
    y, e = ref.turn(x, pos, f, interleaved)
    a = x[..., :8:2] + 1j * x[..., 1:8:2] if interleaved else x[..., :4] + 1j * x[..., 4:8]
    w = a * np.exp(1j * pos[..., None] * f)
    got = y[..., :8:2] + 1j * y[..., 1:8:2] if interleaved else y[..., :4] + 1j * y[..., 4:8]
    assert np.allclose(got, w, rtol=1e-12, atol=1e-12) and (y[..., 8:] == x[..., 8:]).all() and (e[..., 8:] == 0).all()


def test_largest_attention_sizes():
    # b * Hk * ceil(L * Hq / Hk / 16) up to 2^23
    assert ssd.ssd_attn_workspace(1 << 16, 1, 128, 128, 64) == 0
    assert ssd.ssd_attn_workspace(1 << 16, 1, 129, 129, 64) == -1
    assert ssd.ssd_attn_workspace(1 << 16, 16, 128, 128, 64) == 0
    assert ssd.ssd_attn_workspace(1 << 16, 17, 128, 128, 64) == -1
    assert ssd.ssd_attn_workspace(1, 1 << 24, 8, 8, 64) == 0
    assert ssd.ssd_attn_workspace(1, 1 << 24, 9, 9, 64) == -1
    assert ssd.ssd_attn_workspace(1, 1, 1 << 16, 1, 64) > 0
    assert ssd.ssd_attn_workspace(1, 1, 1 << 17, 1, 64) == -1
