"""The cache's append on the GPU against its definition in 64 bits: every place of
both caches, those that nothing is stored to among them."""
import sys

import numpy as np
import pytest
import torch

import attn_ref as ref
from mamba_ssd_scan_05_amd import ssd

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF, F32 = torch.bfloat16, torch.float32


def say(*a):
    print(*a, file=sys.stderr, flush=True)


def num(t):
    return t.float().cpu().double().numpy()


def check(name, got, want, bound):
    half = torch.finfo(got.dtype).eps / 2
    got = num(got)
    tol = bound + half * (np.abs(want) + bound) + 1e-37
    bad = ~(np.abs(got - want) <= tol)
    assert not bad.any(), "%s: %d of %d beyond the bound, worst %.3g of it at %s" % (
        name, bad.sum(), bad.size, np.nanmax(np.abs(got - want) / tol), np.argwhere(bad)[0])


def make(b, L, Hq, Hk, N, npair, page, dtype, layout="dense", ctx=0, pool="apart", seed=1):
    g = torch.Generator().manual_seed(seed)
    n = lambda *s: torch.randn(s, generator=g)  # noqa: E731
    if layout == "fused":
        proj = (3 * n(b, L, Hq + 2 * Hk, N)).to(dtype).to(DEV)
        q, k, v = proj[:, :, :Hq], proj[:, :, Hq:Hq + Hk], proj[:, :, Hq + Hk:]
    elif layout == "offset":
        proj = n(b, L, (Hq + 2 * Hk) * N + 9).to(dtype).to(DEV)
        q = proj[..., 3:3 + Hq * N].unflatten(-1, (Hq, N))
        k = proj[..., 5 + Hq * N:5 + (Hq + Hk) * N].unflatten(-1, (Hk, N))
        v = proj[..., 9 + (Hq + Hk) * N:].unflatten(-1, (Hk, N))
    elif layout == "heads_first":
        q, k, v = (n(b, H, L, N).to(dtype).to(DEV).transpose(1, 2) for H in (Hq, Hk, Hk))
    else:
        q, k, v = (n(b, L, H, N).to(dtype).to(DEV) for H in (Hq, Hk, Hk))
    start = torch.tensor([(ctx * (3 * i + 1)) // (3 * b) for i in range(b)], dtype=torch.int32)
    width = (ctx + L + page - 1) // page + 1
    pages = b * width + 3
    table = torch.randperm(pages, generator=g)[:b * width].view(b, width).to(torch.int32)
    if pool == "apart":
        kc, vc = (torch.full((pages, page, Hk, N), 7.0, dtype=dtype, device=DEV) for _ in range(2))
    elif pool == "halves":
        both = torch.full((pages, 2, page, Hk, N), 7.0, dtype=dtype, device=DEV)
        kc, vc = both[:, 0], both[:, 1]
    else:  # heads before tokens
        kc, vc = (torch.full((pages, Hk, page, N), 7.0, dtype=dtype, device=DEV).transpose(1, 2) for _ in range(2))
    freqs = (10000.0 ** (-torch.arange(npair, dtype=torch.float64) / max(npair, 1))).float() if npair else None
    return dict(q=q, k=k, v=v, freqs=freqs, table=table, start=start, kc=kc, vc=vc)


def expect(t, tokens, interleaved, kc0, vc0):
    """The caches and q_out after the append, and bounds, from their contents before."""
    f = None if t["freqs"] is None else t["freqs"].double().numpy()
    q, k, v = num(t["q"]), num(t["k"]), num(t["v"])
    b, L = k.shape[:2]
    pages, page = t["kc"].shape[:2]
    kc, vc, ek = num(kc0), num(vc0), np.zeros(t["kc"].shape)
    qo, eq = np.full(q.shape, 9.0), np.zeros(q.shape)
    table, start = t["table"].cpu().numpy(), t["start"].cpu().numpy().astype(np.int64)
    for i in range(b):
        for s in range(L if tokens is None else min(max(int(tokens[i]), 0), L)):
            p = start[i] + s
            qo[i, s], eq[i, s] = ref.turn(q[i, s], p, f, interleaved)
            if 0 <= p < table.shape[1] * page and 0 <= table[i, p // page] < pages:
                at = (table[i, p // page], p % page)
                kc[at], ek[at] = ref.turn(k[i, s], p, f, interleaved)
                vc[at] = v[i, s]
    return kc, ek, vc, qo, eq


def run_and_check(t, tokens=None, interleaved=False, with_q=True):
    tok = None if tokens is None else torch.tensor(tokens, dtype=torch.int32, device=DEV)
    d = {k: v.to(DEV) if isinstance(v, torch.Tensor) else v for k, v in t.items()}
    kc, ek, vc, qo, eq = expect(t, tokens, interleaved, t["kc"], t["vc"])
    q_out = torch.full_like(t["q"], 9.0, memory_format=torch.contiguous_format) if with_q else None
    got = ssd.ssd_kv_append(d["k"], d["v"], d["kc"], d["vc"], d["table"], d["start"], q=d["q"] if with_q else None,
                            freqs=d["freqs"], tokens=tok, interleaved=interleaved, q_out=q_out)
    torch.cuda.synchronize()
    assert got is q_out
    check("k_cache", t["kc"], kc, ek)
    assert np.array_equal(num(t["vc"]), vc), "v_cache"
    untouched = ek.max(-1) == 0 if t["freqs"] is not None else np.zeros(ek.shape[:-1], bool)
    assert np.array_equal(num(t["kc"])[untouched], kc[untouched]), "k_cache beside the new tokens"
    if with_q:
        check("q_out", q_out, qo, eq)


CASES = [
    # b, L, Hq, Hk, N, npair, page, layout, ctx, pool
    (1, 1, 1, 1, 8, 4, 1, "dense", 0, "apart"),
    (1, 1, 4, 1, 16, 8, 16, "dense", 5000, "apart"),
    (2, 3, 5, 1, 24, 4, 3, "dense", 10, "halves"),
    (3, 17, 3, 3, 32, 16, 5, "fused", 100, "apart"),
    (1, 65, 2, 1, 40, 0, 7, "dense", 0, "heads"),
    (2, 33, 7, 7, 64, 32, 16, "heads_first", 40, "apart"),
    (1, 9, 6, 2, 80, 20, 24, "offset", 4096, "heads"),
    (32, 1, 32, 8, 128, 64, 16, "fused", 300, "apart"),
    (1, 300, 1, 1, 128, 64, 64, "dense", 129, "halves"),
    (2, 11, 9, 3, 192, 32, 100, "fused", 1000, "apart"),
    (2, 13, 2, 1, 256, 128, 256, "offset", 255, "apart"),
]


@pytest.mark.parametrize("dtype", [F32, BF], ids=["f32", "bf16"])
@pytest.mark.parametrize("interleaved", [False, True], ids=["halves", "adjacent"])
@pytest.mark.parametrize("case", CASES, ids=["b%d_L%d_Hq%d_Hk%d_N%d_p%d_page%d_%s" % c[:8] for c in CASES])
def test_append(case, interleaved, dtype):
    b, L, Hq, Hk, N, npair, page, layout, ctx, pool = case
    say("append", case, interleaved, dtype)
    t = make(b, L, Hq, Hk, N, npair, page, dtype, layout, ctx, pool)
    run_and_check(t, interleaved=interleaved)


@pytest.mark.parametrize("dtype", [F32, BF], ids=["f32", "bf16"])
def test_rows_of_several_lengths(dtype):
    t = make(6, 9, 4, 2, 64, 16, 8, dtype, "fused", 50)
    run_and_check(t, tokens=[0, 1, 9, 5, -3, 100])
    run_and_check(t, tokens=[9, 0, 0, 0, 0, 2], interleaved=True)


def test_keys_only_and_no_turn():
    t = make(3, 5, 4, 2, 32, 16, 4, BF, ctx=9)
    run_and_check(t, with_q=False)
    t = make(3, 5, 4, 2, 32, 0, 4, F32, ctx=9)
    run_and_check(t, tokens=[5, 2, 0])


def test_bad_pages_and_positions_outside():
    # entries that name no page, positions before and behind what the table covers
    t = make(5, 12, 2, 2, 32, 8, 4, F32, ctx=8)
    t["table"][0, 1], t["table"][1, 2], t["table"][2, 0] = -1, 1 << 30, t["kc"].shape[0]
    t["start"][3], t["start"][4] = -5, t["table"].shape[1] * 4 - 3
    run_and_check(t)
    t["start"][3], t["start"][4] = -(1 << 31), (1 << 31) - 1
    run_and_check(t, tokens=[12, 3, 12, 12, 12])


def test_values_are_moved_bit_by_bit():
    for dtype, bits in ((BF, torch.int16), (F32, torch.int32)):
        for layout in ("dense", "offset"):
            t = make(1, 40, 2, 2, 32, 0, 16, dtype, layout)
            info = torch.iinfo(bits)
            raw = torch.randint(info.min, info.max, (1, 40, 2, 32), dtype=bits, device=DEV)
            t["v"].copy_(raw.view(dtype))
            t["v"].view(bits)[0, :4, 0, :2] = raw[0, :4, 0, :2] | (0x7F80 if bits == torch.int16 else 0x7F800000)
            want = t["v"].clone().view(bits)
            d = {k: x.to(DEV) for k, x in t.items() if isinstance(x, torch.Tensor)}
            ssd.ssd_kv_append(d["k"], d["v"], d["kc"], d["vc"], d["table"], d["start"])
            at = d["table"][0].long()[torch.arange(40, device=DEV) // 16] * 16 + torch.arange(40, device=DEV) % 16
            assert torch.equal(t["vc"].view(bits).flatten(0, 1)[at], want[0]), (dtype, layout)
            assert torch.equal(t["kc"].view(bits).flatten(0, 1)[at], t["k"].contiguous().view(bits)[0])


def test_far_positions():
    # the angles of positions up to 2^30, to fp32
    t = make(2, 4, 2, 1, 64, 32, 1 << 20, F32, ctx=0)
    t["kc"], t["vc"] = (torch.full((2, 1 << 20, 1, 64), 7.0, device=DEV) for _ in range(2))
    t["table"] = torch.full((2, 1 << 10), -1, dtype=torch.int32)
    t["table"][0, 1023], t["table"][1, 511] = 1, 0
    t["start"] = torch.tensor([(1 << 30) - 4, (1 << 29) - 3], dtype=torch.int32)
    d = {k: x.to(DEV) for k, x in t.items() if isinstance(x, torch.Tensor)}
    qo = ssd.ssd_kv_append(d["k"], d["v"], d["kc"], d["vc"], d["table"], d["start"], q=d["q"], freqs=d["freqs"])
    f = t["freqs"].double().numpy()
    for i in range(2):
        pos = int(t["start"][i]) + np.arange(4)
        y, e = ref.turn(num(t["q"])[i], pos[:, None], f, False)
        check("q_out", qo[i], y, e)
        y, e = ref.turn(num(t["k"])[i], pos[:, None], f, False)
        n = 4 if i == 0 else 3  # the last token of row 1 begins a page that is not dealt out
        check("k", d["kc"][1 - i, (1 << 20) - n:], y[:n], e[:n])


def test_replayed_graph_and_another_stream():
    t = make(4, 1, 4, 2, 64, 32, 16, BF, "fused", 60)
    d = {k: x.to(DEV) for k, x in t.items() if isinstance(x, torch.Tensor)}
    q_out = torch.empty_like(d["q"], memory_format=torch.contiguous_format)

    def call():
        ssd.ssd_kv_append(d["k"], d["v"], d["kc"], d["vc"], d["table"], d["start"], q=d["q"], freqs=d["freqs"], q_out=q_out)
    call()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for k in range(4):
        d["start"].add_(1)
        t["start"] = d["start"]
        d["kc"].fill_(7.0), d["vc"].fill_(7.0)
        d["q"].mul_(-1.0), d["k"].add_(0.5)
        kc, ek, vc, qo, eq = expect(t, None, False, d["kc"], d["vc"])
        graph.replay()
        torch.cuda.synchronize()
        check("k_cache", d["kc"], kc, ek)
        assert np.array_equal(num(d["vc"]), vc)
        check("q_out", q_out, qo, eq)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    want = d["kc"].clone()
    d["kc"].fill_(7.0)
    s.wait_stream(torch.cuda.current_stream())
    got = ssd.ssd_kv_append(d["k"], d["v"], d["kc"], d["vc"], d["table"], d["start"], q=d["q"], freqs=d["freqs"],
                            stream=s.cuda_stream)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(got, q_out) and torch.equal(d["kc"], want)
