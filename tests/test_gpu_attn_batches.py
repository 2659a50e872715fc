"""Attention over the paged cache for batches that take each of the plans: so many rows
that none is cut into pieces, more rows than a wave has lanes, rows that pass the 1024 keys
whose places are found at once; and odd values in queries and scores.  Some rows of each
are compared (the others run beside them)."""
import sys

import numpy as np
import pytest
import torch

from mamba_ssd_scan_05_amd import ssd
from test_gpu_attn import BF, DEV, F32, Batch, check

pytestmark = pytest.mark.gpu


def some(batch, rows, scale=None, window=0, step=False):
    scale = float(np.float32(batch.N ** -0.5 if scale is None else scale))
    got, lse = batch.call(scale, window, step)
    torch.cuda.synchronize()
    part = object.__new__(Batch)
    part.__dict__.update(batch.__dict__, b=len(rows), starts=[batch.starts[i] for i in rows],
                         counts=[batch.counts[i] for i in rows], k=[batch.k[i] for i in rows],
                         v=[batch.v[i] for i in rows], q=batch.q[rows], table=batch.table[rows])
    want, wl, eo, el = part.expect(scale, window)
    check("out", got[rows], want, eo)
    check("lse", lse[rows], wl, el)


CASES = [
    # rows, start up to, L, Hq, Hk, N, page, window
    (1030, 45, 1, 16, 8, 16, 16, 0),       # no pieces, one token
    (1030, 45, 1, 16, 8, 24, 7, 20),
    (64, 40, 20, 8, 8, 32, 16, 0),         # no pieces, several tokens
    (64, 2300, 17, 8, 8, 64, 48, 0),       # and past 1024 keys
    (64, 2300, 17, 8, 8, 40, 10, 0),
    (1024, 1500, 1, 8, 8, 8, 16, 0),       # one token past 1024 keys
    (1024, 1500, 1, 8, 8, 8, 6, 1200),
    (70, 900, 5, 4, 1, 64, 16, 0),         # pieces of more rows than a wave has lanes
    (70, 900, 5, 4, 1, 200, 9, 300),
    (300, 400, 1, 3, 1, 128, 32, 0),
    (2, 200, 9, 2, 2, 256, 16, 0),
]


@pytest.mark.parametrize("dtype", [F32, BF], ids=["f32", "bf16"])
@pytest.mark.parametrize("case", CASES, ids=["b%d_s%d_L%d_Hq%d_Hk%d_N%d_page%d_w%d" % c for c in CASES])
def test_batches(case, dtype):
    b, ctx, L, Hq, Hk, N, page, window = case
    print("batch", case, dtype, file=sys.stderr, flush=True)
    starts = [(ctx * ((37 * i) % 101)) // 100 for i in range(b)]
    counts = [L if i % 5 else (i // 5) % (L + 1) for i in range(b)] if L > 1 else [1] * b
    t = Batch(starts, counts, L, Hq, Hk, N, page, dtype, seed=b + L, spare=0)
    rows = sorted({0, 1, b - 1, b // 2, min(b - 1, 64), int(np.argmax(starts)), int(np.argmin(starts)), b // 3})
    some(t, rows, window=window, step=L == 1)


@pytest.mark.parametrize("dtype", [F32, BF], ids=["f32", "bf16"])
@pytest.mark.parametrize("L", [3, 40])
def test_an_odd_query_stays_with_itself(L, dtype):
    t = Batch([90], [L], L, 4, 2, 64, 16, dtype, seed=2)
    want, wl = t.call(0.125, 0)
    for bad in (float("nan"), float("inf")):
        q = t.q.clone()
        q[0, 1, 2, 7] = bad
        got, gl = t.call(0.125, 0, q=q.to(DEV))
        assert not torch.isfinite(got[0, 1, 2].float()).any()
        for o, w in ((got, want), (gl, wl)):
            o, w = o.clone(), w.clone()
            o[0, 1, 2] = w[0, 1, 2] = 0
            assert torch.equal(o, w)


@pytest.mark.parametrize("dtype", [F32, BF], ids=["f32", "bf16"])
@pytest.mark.parametrize("L", [1, 30])
def test_scores_of_minus_infinity(L, dtype):
    # keys with an infinity against queries above 0: weight 0, as if they were not there;
    # where nothing else is seen, out 0 and lse -infinity
    t = Batch([70, 0], [L, L], L, 4, 2, 32, 16, dtype, seed=3)
    t.q = t.q.abs() + 0.5
    for i, j in ((0, 0), (0, 33), (0, 70), (1, 0)):
        t.kc[int(t.table[i, j // 16]), j % 16, :, 3] = float("-inf")
        t.k[i][j] = float("nan")  # not seen, says the reference
    t.check(step=L == 1)
    out, lse = t.call(0.2, 0, step=L == 1)
    assert (out[1, 0] == 0).all() and (lse[1, 0] == float("-inf")).all()


def test_two_host_threads_at_once():
    import threading
    ts = [Batch([500 + 300 * k, 40], [1, 1], 1, 8, 2, 128, 16, BF, seed=k) for k in range(2)]
    want = [t.call(0.1, 0, True) for t in ts]
    torch.cuda.synchronize()
    bad = []

    def work(k):
        s = torch.cuda.Stream()
        with torch.cuda.stream(s):
            for _ in range(50):
                out, lse = ts[k].call(0.1, 0, True)
                s.synchronize()
                if not (torch.equal(out, want[k][0]) and torch.equal(lse, want[k][1])):
                    bad.append(k)
    th = [threading.Thread(target=work, args=(k,)) for k in range(2)]
    [x.start() for x in th]
    [x.join() for x in th]
    assert not bad


def test_small_tables_need_little():
    # the workspace does not depend on the table; the same call with a wider one
    t = Batch([300, 20], [1, 1], 1, 4, 2, 64, 16, F32, spare=0)
    a, la = t.call(0.1, 0, True)
    t.table = torch.nn.functional.pad(t.table, (0, 3000), value=-1)
    c, lc = t.call(0.1, 0, True)
    assert torch.equal(a, c) and torch.equal(la, lc)
    s = torch.tensor([300, 20], dtype=torch.int32, device=DEV)
    wide = torch.full((2, 4000), 7, dtype=torch.int32, device=DEV)
    wide[:, 100:100 + t.table.shape[1]] = t.table.to(DEV)
    d = ssd.ssd_attn_step(t.q[:, 0].to(DEV), t.kc, t.vc, wide[:, 100:100 + t.table.shape[1]], s, scale=0.1)
    assert torch.equal(d, a[:, 0])


@pytest.mark.parametrize("dtype", [F32, BF], ids=["f32", "bf16"])
@pytest.mark.parametrize("window", [0, 1100])
def test_a_long_row_among_short_ones(window, dtype):
    # workgroups enough without pieces, but the table allows a row many times its new tokens
    starts = [5000 if i == 9 else 30 + i for i in range(32)]
    t = Batch(starts, [70 - i % 3 for i in range(32)], 70, 32, 8, 32, 16, dtype, seed=4, spare=0)
    some(t, [0, 8, 9, 10, 31], window=window)


@pytest.mark.parametrize("dtype", [F32, BF], ids=["f32", "bf16"])
def test_rows_of_several_tiles_uncut(dtype):
    # no pieces, though below 8192 workgroups; keys past the 1024 whose places are found at once
    t = Batch([800 - 9 * i for i in range(22)], [300 - i for i in range(22)], 300, 16, 8, 24, 16, dtype, seed=5, spare=0)
    some(t, [0, 1, 21])


@pytest.mark.parametrize("dtype", [F32, BF], ids=["f32", "bf16"])
def test_a_long_row_among_a_thousand(dtype):
    # 8240 workgroups without pieces; the table allows more keys than one should walk alone
    starts = [4500 if i == 700 else 20 + i % 30 for i in range(1030)]
    t = Batch(starts, [1] * 1030, 1, 8, 8, 16, 16, dtype, seed=6, spare=0)
    some(t, [0, 1, 699, 700, 701, 1029], step=True)


@pytest.mark.parametrize("dtype", [F32, BF], ids=["f32", "bf16"])
@pytest.mark.parametrize("b", [6, 70])
def test_pieces_of_uneven_rows(b, dtype):
    # as many keys as make pieces of few rounds: those of uneven rows are halved
    top = 5500 if b == 6 else 450
    starts = [top * (i % 6 + 1) // 6 - 1 if i % 6 else 2 * top - 1 for i in range(b)]
    t = Batch(starts, [1] * b, 1, 16, 8, 256, 64, dtype, seed=7, spare=0)
    some(t, sorted({0, 1, 5, b // 2, b - 1}), step=True)
